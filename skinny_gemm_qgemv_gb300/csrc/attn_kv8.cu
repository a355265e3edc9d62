// Attention of a step's query tokens over the paged 8-bit key/value cache.
//
// attn_kv8_plain_kernel: one CTA per (query token, query head), four warps that
// take the context's tokens in turn; a lane holds D / 32 (rounded up to words)
// elements of q and of the output. One pass with the running maximum and sum of
// the softmax.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kPlainWarps = 4;

template <int FMT>
__global__ void __launch_bounds__(32 * kPlainWarps) attn_kv8_plain_kernel(AttnArgs a) {
  __shared__ float sm_m[kPlainWarps], sm_l[kPlainWarps], sm_o[kPlainWarps][256];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x, hq = blockIdx.y, h = hq / (a.Hq / a.Hkv);
  if (t < a.cu_q[0] || t >= a.cu_q[a.R]) return;
  int r = 0;
  for (int hi = a.R; hi - r > 1;) {
    const int mid = (r + hi) >> 1;
    if (a.cu_q[mid] <= t)
      r = mid;
    else
      hi = mid;
  }
  const int n = a.cu_q[r + 1] - a.cu_q[r];
  int ctx = max(a.ctx_lens[r], 0);
  if (ctx > a.max_blocks * a.bs) {
    if (threadIdx.x == 0) report_error(a.err, kErrKvLength);
    ctx = a.max_blocks * a.bs;
  }
  const int base = ctx - n;  // first query token's position
  const bool tree = a.tree && n <= 32;
  const uint32_t bits = tree ? a.tree[t] : 0u;
  const int end = tree ? ctx : min(ctx, base + (t - a.cu_q[r]) + 1);
  const int words = a.D / 4;
  float q[2][4] = {}, o[2][4] = {};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int i = lane + 32 * w;
    if (i < words) {
      const uint2 v = *reinterpret_cast<const uint2*>(a.q + t * a.q_stride + (size_t)hq * a.D + 4 * i);
      q[w][0] = bf16_bits_to_f32(v.x & 0xFFFFu), q[w][1] = bf16_bits_to_f32(v.x >> 16);
      q[w][2] = bf16_bits_to_f32(v.y & 0xFFFFu), q[w][3] = bf16_bits_to_f32(v.y >> 16);
    }
  }
  float m = -INFINITY, l = 0.f;
  for (int tok = warp; tok < end; tok += kPlainWarps) {
    if (tree && tok >= base && !(tok - base < 32 && (bits >> (tok - base) & 1u))) continue;
    const int blk = a.table[(size_t)r * a.max_blocks + tok / a.bs];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0) report_error(a.err, kErrKvBlock);
      continue;
    }
    const size_t page = (size_t)blk * a.Hkv + h;
    const size_t at = (page * a.bs + tok % a.bs) * a.D;
    const float ks = a.scales[2 * page], vs = a.scales[2 * page + 1];
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int i = lane + 32 * w;
      if (i < words) {
        float k0, k1, k2, k3;
        kv8_decode4<FMT>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.k_cache) + at + 4 * i), k0, k1,
                         k2, k3);
        s += q[w][0] * k0 + q[w][1] * k1 + q[w][2] * k2 + q[w][3] * k3;
      }
    }
    s = warp_sum(s) * (ks * a.scale_log2);
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int i = lane + 32 * w;
      if (i < words) {
        float v0, v1, v2, v3;
        kv8_decode4<FMT>(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v_cache) + at + 4 * i), v0, v1,
                         v2, v3);
        const float pv = p * vs;
        o[w][0] = o[w][0] * c + pv * v0;
        o[w][1] = o[w][1] * c + pv * v1;
        o[w][2] = o[w][2] * c + pv * v2;
        o[w][3] = o[w][3] * c + pv * v3;
      }
    }
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * w < words) sm_o[warp][4 * (lane + 32 * w) + j] = o[w][j];
  __syncthreads();
  float mm = sm_m[0];
  for (int w = 1; w < kPlainWarps; ++w) mm = fmaxf(mm, sm_m[w]);
  float ll = 0.f, f[kPlainWarps];
  for (int w = 0; w < kPlainWarps; ++w) {
    f[w] = sm_m[w] == -INFINITY ? 0.f : exp2f(sm_m[w] - mm);
    ll += sm_l[w] * f[w];
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + ((size_t)t * a.Hq + hq) * a.D);
  for (int i = threadIdx.x; i < a.D / 2; i += blockDim.x) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kPlainWarps; ++w) x += f[w] * sm_o[w][2 * i], y += f[w] * sm_o[w][2 * i + 1];
    const bool none = mm == -INFINITY;  // no token seen
    out[i] = f32_to_bf16x2(none ? 0.f : x / ll, none ? 0.f : y / ll);
  }
}

}  // namespace

size_t attn_kv8_workspace_size(int, int, int) { return 0; }

cudaError_t launch_attn_kv8(const AttnArgs& a, int format, cudaStream_t stream, bool pdl) {
  auto k = format == QG_KV_I8 ? attn_kv8_plain_kernel<QG_KV_I8> : attn_kv8_plain_kernel<QG_KV_E4M3>;
  return launch_kernel(k, dim3(a.T, a.Hq), dim3(32 * kPlainWarps), 0, stream, pdl, a);
}

}  // namespace qg
