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
// Many rows are bound by HBM (4096 rows of 7168, bf16 to int8 codes: 205 MB in
// 37 us, 5.6 TB/s; to bf16 235 MB in 35 us), few rows by the launch and one trip through load, two
// reductions and store (one row of 4096: 3.7 us).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

// elements 8i .. 8i + 7 of a bf16 or fp32 array as loaded; converted apart from the load, so that a thread's loads
// are all on the way before the first is waited for
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* p, size_t i) {
  Raw8<F32> r;
  const uint4* s = static_cast<const uint4*>(p) + (F32 ? 2 * i : i);
  r.v[0] = s[0];
  if (F32) r.v[F32 ? 1 : 0] = s[1];
  return r;
}
template <bool F32>
__device__ __forceinline__ void to_f32(const Raw8<F32>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[F32].x, r.v[F32].y, r.v[F32].z, r.v[F32].w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __uint_as_float(F32 ? w[j] : j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
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

// C: steps of 8 elements per thread (C * blockDim.x * 8 >= K); XF, RF: x and the
// residual are fp32. All of a thread's loads are issued before anything is
// stored (residual_out may be residual, so the compiler cannot move a load over
// a store by itself).
template <int C, int THREADS, bool I8, bool XF, bool RF>
__global__ void __launch_bounds__(THREADS) rmsnorm_kernel(const void* x, const void* res,
                                                          const void* __restrict__ w, int w_f32, float eps,
                                                          const uint32_t* __restrict__ sign_bits, int K, void* res_out,
                                                          void* __restrict__ out, float* __restrict__ scale) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int n8 = K / 8;
  const size_t row = (size_t)blockIdx.x * n8;
  Raw8<XF> xr[C];
  Raw8<RF> rr[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      xr[c] = load8<XF>(x, row + i);
      if (res) rr[c] = load8<RF>(res, row + i);
    }
  }
  // the first step's weights too (a row of few steps is all latency)
  Raw8<true> w0;
  if (threadIdx.x < n8) {
    const uint4* s = static_cast<const uint4*>(w) + (w_f32 ? 2 : 1) * threadIdx.x;
    w0.v[0] = s[0];
    if (w_f32) w0.v[1] = s[1];
  }
  float h[C][8], ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      to_f32<XF>(xr[c], h[c]);
      if (res) {
        float r[8];
        to_f32<RF>(rr[c], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[c][j] += r[j];
      }
      if (res_out) {
        if (RF) {
          float4* d = static_cast<float4*>(res_out) + 2 * (row + i);
          d[0] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
          d[1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
        } else {
          uint32_t b[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            b[j] = f32_to_bf16x2(h[c][2 * j], h[c][2 * j + 1]);
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
      if (w_f32) {
        to_f32<true>(c == 0 ? w0 : load8<true>(w, i), g);
      } else {
        Raw8<false> b;
        b.v[0] = w0.v[0];
        if (c > 0) b = load8<false>(w, i);
        to_f32<false>(b, g);
      }
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
        static_cast<uint4*>(out)[row + i] = make_uint4(f32_to_bf16x2(h[c][0], h[c][1]), f32_to_bf16x2(h[c][2], h[c][3]),
                                                       f32_to_bf16x2(h[c][4], h[c][5]), f32_to_bf16x2(h[c][6], h[c][7]));
      }
    }
  }
  if (!I8) return;
  amax = cta_reduce<true>(amax, part[1]);
  const float s = __fdiv_rn(amax, 127.f);
  const float inv = __frcp_rn(s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * blockDim.x;
    if (i < n8) {
      static_cast<uint2*>(out)[row + i] = s > 0.f ? kv8_quantize8<QG_KV_I8>(h[c], s, inv) : make_uint2(0u, 0u);
    }
  }
}

template <int C, int THREADS, bool I8>
cudaError_t launch_types(const NormArgs& a, int threads, cudaStream_t stream, bool pdl) {
  auto k = a.x_f32 ? (a.res_f32 ? rmsnorm_kernel<C, THREADS, I8, true, true> : rmsnorm_kernel<C, THREADS, I8, true, false>)
                   : (a.res_f32 ? rmsnorm_kernel<C, THREADS, I8, false, true>
                                : rmsnorm_kernel<C, THREADS, I8, false, false>);
  return launch_kernel(k, dim3(a.M), dim3(threads), 0, stream, pdl, a.x, a.res, a.w, a.w_f32, a.eps, a.sign_bits, a.K,
                       a.res_out, a.out, a.scale);
}

template <bool I8>
cudaError_t launch(const NormArgs& a, cudaStream_t stream, bool pdl) {
  const int n8 = a.K / 8;
  auto threads = [&](int c) { return ((n8 + c - 1) / c + 31) / 32 * 32; };
  // Few rows: as many threads as a row has steps, for latency. Many rows (four CTAs an SM and more) of up to 8192
  // elements: several steps per thread, so that more bytes are on the way per SM (4096 rows of 7168 bf16, int8 codes:
  // 57 -> 37 us).
  if (n8 <= 1024 && a.M >= 4 * device_sm_count())
    return n8 <= 512 ? launch_types<2, 256, I8>(a, threads(2), stream, pdl)
                     : launch_types<4, 256, I8>(a, threads(4), stream, pdl);
  if (n8 <= 1024) return launch_types<1, 1024, I8>(a, threads(1), stream, pdl);
  if (n8 <= 2048) return launch_types<2, 1024, I8>(a, threads(2), stream, pdl);
  return launch_types<4, 1024, I8>(a, threads(4), stream, pdl);
}

}  // namespace

cudaError_t launch_rmsnorm(const NormArgs& a, cudaStream_t stream, bool pdl) {
  return a.scale ? launch<true>(a, stream, pdl) : launch<false>(a, stream, pdl);
}

}  // namespace qg
