// Residual addition + RMS norm, as bf16 or as int8 codes with a scale per row.
//
//   h = x + residual (stored in the residual's type), y = (h r) w with
//   r = 1 / sqrt(mean(h^2) + eps); then bf16(y), or z = y or its block-32
//   randomized Hadamard transform and s = max|z| / 127, q = rint(z / s).
//
// GB300 mapping: one CTA per row. A row is read once and stays in registers
// (8 consecutive elements per thread and step, 16- or 32-byte loads) through
// both reductions, the transform and the quantizer, so the traffic is the
// algorithmic one. A 32-block of the transform is four neighbouring lanes: the
// butterflies of span 1, 2, 4 stay in a thread, 8 and 16 are two shuffles.
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

// elements 8i .. 8i + 7 of a bf16 or fp32 array, as fp32
__device__ __forceinline__ void load8(const void* p, int f32, size_t i, float (&v)[8]) {
  if (f32) {
    const float4* s = static_cast<const float4*>(p) + 2 * i;
    const float4 a = s[0], b = s[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = static_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// two fp32 rounded to nearest even, as a bf16 pair (lo in the low half)
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// reduction over the CTA: every thread gets the result; `part` has 32 floats
// and is not reused by the caller
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < nw ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  return v;
}

// C: steps of 8 elements per thread (C * blockDim.x * 8 >= K)
template <int C, bool I8>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const void* __restrict__ x, int x_f32, const void* res,
                                                       int res_f32, const void* __restrict__ w, int w_f32, float eps,
                                                       const uint32_t* __restrict__ sign_bits, int K, void* res_out,
                                                       void* __restrict__ out, float* __restrict__ scale) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int n8 = K / 8;
  const size_t row = (size_t)blockIdx.x * n8;
  float h[C][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      load8(x, x_f32, row + i, h[c]);
      if (res) {
        float r[8];
        load8(res, res_f32, row + i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
      }
      if (res_out) {
        if (res_f32) {
          float4* d = static_cast<float4*>(res_out) + 2 * (row + i);
          d[0] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
          d[1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
        } else {
          uint32_t b[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b[j] = bf16x2(h[c][2 * j], h[c][2 * j + 1]);
            h[c][2 * j] = __uint_as_float(b[j] << 16);
            h[c][2 * j + 1] = __uint_as_float(b[j] & 0xFFFF0000u);
          }
          static_cast<uint4*>(res_out)[row + i] = make_uint4(b[0], b[1], b[2], b[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += h[c][j] * h[c][j];
    }
  }
  ss = cta_reduce<false>(ss, part[0]);
  const float r = __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)K), eps));
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    // lanes of one 32-block are in or out of the row together (K % 32 == 0)
    if (i < n8) {
      float g[8];
      load8(w, w_f32, i, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = __fmul_rn(__fmul_rn(h[c][j], r), g[j]);
      if (I8) {
        if (sign_bits) {
          const uint32_t sb = sign_bits[i >> 2] >> (8 * (i & 3));
#pragma unroll
          for (int j = 0; j < 8; ++j) h[c][j] = __uint_as_float(__float_as_uint(h[c][j]) ^ ((sb >> j & 1u) << 31));
#pragma unroll
          for (int s = 1; s < 8; s <<= 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (!(j & s)) {
                const float a = h[c][j], b = h[c][j + s];
                h[c][j] = __fadd_rn(a, b);
                h[c][j + s] = __fsub_rn(a, b);
              }
            }
          }
          const unsigned quad = 0xFu << (threadIdx.x & 28);
#pragma unroll
          for (int s = 1; s < 4; s <<= 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float p = __shfl_xor_sync(quad, h[c][j], s);
              h[c][j] = (threadIdx.x & s) ? __fsub_rn(p, h[c][j]) : __fadd_rn(h[c][j], p);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(h[c][j]));
      } else {
        static_cast<uint4*>(out)[row + i] = make_uint4(bf16x2(h[c][0], h[c][1]), bf16x2(h[c][2], h[c][3]),
                                                       bf16x2(h[c][4], h[c][5]), bf16x2(h[c][6], h[c][7]));
      }
    }
  }
  if (!I8) return;
  amax = cta_reduce<true>(amax, part[1]);
  const float s = __fdiv_rn(amax, 127.f);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      uint32_t o[2] = {0u, 0u};
      if (s > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = fminf(fmaxf(rintf(__fdiv_rn(h[c][j], s)), -127.f), 127.f);
          o[j >> 2] |= ((uint32_t)(int)t & 0xFFu) << (8 * (j & 3));
        }
      }
      static_cast<uint2*>(out)[row + i] = make_uint2(o[0], o[1]);
    }
  }
}

template <bool I8>
cudaError_t launch(const NormArgs& a, cudaStream_t stream, bool pdl) {
  const int n8 = a.K / 8;
  const int c = n8 <= 1024 ? 1 : n8 <= 2048 ? 2 : 4;
  const int threads = ((n8 + c - 1) / c + 31) / 32 * 32;
  auto k = c == 1 ? rmsnorm_kernel<1, I8> : c == 2 ? rmsnorm_kernel<2, I8> : rmsnorm_kernel<4, I8>;
  return launch_kernel(k, dim3(a.M), dim3(threads), 0, stream, pdl, a.x, a.x_f32, a.res, a.res_f32, a.w, a.w_f32,
                       a.eps, a.sign_bits, a.K, a.res_out, a.out, a.scale);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t stream, bool pdl) {
  return a.scale ? launch<true>(a, stream, pdl) : launch<false>(a, stream, pdl);
}

}  // namespace qg
