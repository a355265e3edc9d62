// Norms of queries and keys for each head with the position rotation, in one pass.
//
//   y = x r w, r = 1 / sqrt(mean(x^2) + eps) over a head's D elements (or y = x);
//   pair i of the first `rot` elements turns by a = position[axis(i)] inv_freq[i]:
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a).
//
// GB300 mapping: a head is 16 or 32 lanes' with four consecutive elements a lane
// (eight for heads of more than 128), so it stays in registers from one load to one
// store: HBM bounds many tokens, launch and one trip of loads a few. The sines of a
// token are formed once for all of its heads, by one thread a pair, into one of two
// tables in shared memory (one barrier a token).
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

constexpr int kThreads = 256, kWarps = kThreads / 32;

// four consecutive elements as loaded, and as fp32
template <bool F32>
struct Quad {
  uint4 v;  // bf16: .x, .y
};
template <bool F32>
__device__ __forceinline__ Quad<F32> load_quad(const void* p, long long i) {
  Quad<F32> r;
  if (F32) {
    r.v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    r.v = make_uint4(w.x, w.y, 0u, 0u);
  }
  return r;
}
template <bool F32>
__device__ __forceinline__ void to_f32(const Quad<F32>& r, float (&f)[4]) {
  if (F32) {
    f[0] = __uint_as_float(r.v.x), f[1] = __uint_as_float(r.v.y);
    f[2] = __uint_as_float(r.v.z), f[3] = __uint_as_float(r.v.w);
  } else {
    f[0] = __uint_as_float(r.v.x << 16), f[1] = __uint_as_float(r.v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(r.v.y << 16), f[3] = __uint_as_float(r.v.y & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void weights4(const void* w, int f32, int at, float (&f)[4]) {
  if (f32) {
    to_f32<true>(load_quad<true>(w, at), f);
  } else {
    to_f32<false>(load_quad<false>(w, at), f);
  }
}

// L: lanes of a head; C: runs of four elements a lane has, 4 L apart; F32: the type of x; UN: heads of a warp at a time
template <bool F32, int L, int C, int UN>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(RopeArgs a) {
  __shared__ float2 turn[2][128];  // (cos, sin) of the token's pairs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int HW = 32 / L;  // heads of a warp's load
  const int ql = lane % L, half = a.rot / 2;
  pdl_wait();
  pdl_launch_dependents();

  // the pair that this thread looks after: the fraction of a turn per position, times 2^64
  unsigned long long step = 0;
  int axis = 0;
  if (threadIdx.x < half) {
    const double t = a.inv_freq[threadIdx.x] * 0.15915494309189533577;  // 1 / (2 pi)
    step = 2ull * (unsigned long long)__double2ll_rn((t - rint(t)) * 9223372036854775808.0);
    axis = a.axis_bits[threadIdx.x >> 4] >> (2 * (threadIdx.x & 15)) & 3u;
  }
  // this lane's weights; its elements past the head count as 0
  float wq[C][4], wk[C][4];
  bool in[C], turns[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = 4 * (ql + L * c);
    in[c] = e < a.D, turns[c] = e < a.rot;
#pragma unroll
    for (int j = 0; j < 4; ++j) wq[c][j] = wk[c][j] = 1.f;
    if (in[c] && a.q_w) weights4(a.q_w, a.w_f32, e, wq[c]);
    if (in[c] && a.k_w) weights4(a.k_w, a.w_f32, e, wk[c]);
  }
  const int heads = a.Hq + a.Hkv, units = (heads + HW - 1) / HW;
  const int u0 = blockIdx.y * kWarps + warp, du = gridDim.y * kWarps;
  const float inv_d = 1.f / (float)a.D;
  const int shift = half / 4;  // quads between the elements of a pair (split halves)

  int b = 0;
#pragma unroll 1
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (a.pos[t] < 0) continue;  // padding (the same for all threads)
    auto head_of = [&](int u) { return u * HW + lane / L; };
    Quad<F32> raw[UN][C];
    auto fetch = [&](int u) {
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        const int h = head_of(u + n * du);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          raw[n][c].v = make_uint4(0u, 0u, 0u, 0u);
          if (h < heads && in[c]) {
            const int e = 4 * (ql + L * c);
            raw[n][c] = h < a.Hq ? load_quad<F32>(a.q, t * a.q_stride + h * a.D + e)
                                 : load_quad<F32>(a.k, t * a.k_stride + (h - a.Hq) * a.D + e);
          }
        }
      }
    };
    fetch(u0);  // on the way while the sines are formed
    if (threadIdx.x < half) {
      const long long p = a.pos[(long long)axis * a.T + t];
      const float half_turns = (float)(long long)(step * (unsigned long long)p) * 0x1p-63f;  // in [-1, 1]
      float s, c;
      sincospif(half_turns, &s, &c);
      turn[b][threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();  // (a table is read right after its barrier, and written again past the next token's)
    // y = x cs + (its partner) sn
    float cs[C][4], sn[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 4 * (ql + L * c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cs[c][j] = 1.f, sn[c][j] = 0.f;
        if (turns[c]) {
          const bool lo = a.interleaved ? j % 2 == 0 : e < half;
          const float2 x = turn[b][a.interleaved ? (e + j) / 2 : lo ? e + j : e + j - half];
          cs[c][j] = x.x, sn[c][j] = lo ? -x.y : x.y;
        }
      }
    }
#pragma unroll 1
    for (int u = u0; u < units; u += UN * du) {
      if (u != u0) fetch(u);
#pragma unroll
      for (int n = 0; n < UN; ++n) {
        const int h = head_of(u + n * du);
        const bool is_q = h < a.Hq;
        float x[C][4];
        float ss = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          to_f32<F32>(raw[n][c], x[c]);
#pragma unroll
          for (int j = 0; j < 4; ++j) ss = fmaf(x[c][j], x[c][j], ss);
        }
        if (a.q_w || a.k_w) {
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
          const bool normed = is_q ? a.q_w != nullptr : a.k_w != nullptr;
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (normed) x[c][j] = x[c][j] * r * (is_q ? wq[c][j] : wk[c][j]);
        }
        float y[C][4];
        if (a.interleaved) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[c][j] = turns[c] ? fmaf(x[c][j], cs[c][j], x[c][j ^ 1] * sn[c][j]) : x[c][j];
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int at = ql + L * c, from = turns[c] ? (at < shift ? at + shift : at - shift) : at;
            const int src = (lane & ~(L - 1)) | (from & (L - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float p = __shfl_sync(0xffffffffu, x[0][j], src);
              if (C == 2) {
                const float p1 = __shfl_sync(0xffffffffu, x[C - 1][j], src);
                if (from >= L) p = p1;
              }
              y[c][j] = turns[c] ? fmaf(x[c][j], cs[c][j], p * sn[c][j]) : x[c][j];
            }
          }
        }
        if (h < heads) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            if (!in[c]) continue;
            const int e = 4 * (ql + L * c);
            const uint2 packed = make_uint2(f32_to_bf16x2(y[c][0], y[c][1]), f32_to_bf16x2(y[c][2], y[c][3]));
            if (is_q) {
              *reinterpret_cast<uint2*>(a.q_out + ((long long)t * a.Hq + h) * a.D + e) = packed;
            } else {
              const long long to = ((long long)t * a.Hkv + h - a.Hq) * a.D + e;
              if (a.k_out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(a.k_out) + to) = make_float4(y[c][0], y[c][1], y[c][2], y[c][3]);
              else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.k_out) + to) = packed;
            }
          }
        }
      }
    }
    b ^= 1;
  }
}

template <bool F32, int L, int C>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream, bool pdl) {
  const int sms = device_sm_count();
  const int units = (a.Hq + a.Hkv + 32 / L - 1) / (32 / L), per = (units + kWarps - 1) / kWarps;
  // few tokens: their heads over several CTAs, a head a warp
  const int split = std::min(per, std::max(1, 2 * sms / a.T));
  const int grid = std::min(a.T, 8 * sms);
  auto k = qk_rope_kernel<F32, L, C, 2>;
  return launch_kernel(k, dim3(grid, split), dim3(kThreads), 0, stream, pdl, a);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t stream, bool pdl) {
  if (a.D <= 64) return a.x_f32 ? launch<true, 16, 1>(a, stream, pdl) : launch<false, 16, 1>(a, stream, pdl);
  if (a.D <= 128) return a.x_f32 ? launch<true, 32, 1>(a, stream, pdl) : launch<false, 32, 1>(a, stream, pdl);
  return a.x_f32 ? launch<true, 32, 2>(a, stream, pdl) : launch<false, 32, 2>(a, stream, pdl);
}

}  // namespace qg
