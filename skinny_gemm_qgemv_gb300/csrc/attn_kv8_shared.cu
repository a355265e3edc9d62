// Attention of requests whose groups share a prefix of the paged 8-bit cache.
//
// With z_j the scores of a row, the sums over the shared prefix P and over the
// request's own tokens S join as
//   m = max(m_P, m_S), out = (2^(m_P - m) l_P o_P + 2^(m_S - m) l_S o_S) /
//                            (2^(m_P - m) l_P + 2^(m_S - m) l_S),
// so the prefix is read once for all query rows of its group instead of once per
// request. Three launches: every request over its own tokens, every group over its
// prefix (no mask: all of it is seen), both leaving a row's maximum, sum and fp32
// output in the workspace, and the joining.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_kv8_mma.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

struct JoinArgs {
  const int32_t *cu_q, *cu_req;
  int R, groups, T, Hq, D;
  const float *own_o, *pre_o;
  const float2 *own_ml, *pre_ml;
  uint16_t* out;
};

constexpr int kJoinThreads = 256;

// true in all threads where the bounds do not ascend within T (the passes have reported it and computed nothing)
__device__ bool bounds_bad(const int32_t* cu, int n, int top) {
  bool bad = false;
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= cu[i] < 0 || cu[i] > cu[i + 1] || cu[i + 1] > top;
  return __syncthreads_or(bad);
}

// A row is a quarter of a warp's (heads of up to 256: 4 to 8 consecutive elements a lane at a time).
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(JoinArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  if (bounds_bad(a.cu_q, a.R, a.T) || bounds_bad(a.cu_req, a.groups, a.R)) return;
  const int t0 = a.cu_q[0], t1 = a.cu_q[a.R], g0 = a.cu_q[a.cu_req[0]], g1 = a.cu_q[a.cu_req[a.groups]];
  const int lanes = 8, per = kJoinThreads / lanes, lane = threadIdx.x % lanes;
  const long long rows = (long long)(t1 - t0) * a.Hq;
#pragma unroll 1
  for (long long i = (long long)blockIdx.x * per + threadIdx.x / lanes; i < rows; i += (long long)gridDim.x * per) {
    const int t = t0 + (int)(i / a.Hq);
    const long long row = (long long)t0 * a.Hq + i;
    const bool shared = t >= g0 && t < g1;
    const float2 s = a.own_ml[row], p = shared ? a.pre_ml[row] : make_float2(kNoMax, 0.f);
    const float m = fmaxf(s.x, p.x);
    float fs = s.y > 0.f ? s.y * ex2(s.x - m) : 0.f, fp = p.y > 0.f ? p.y * ex2(p.x - m) : 0.f;
    // (a sum that is no number makes the row none, as it would alone)
    if (s.y != s.y) fs = s.y;
    if (p.y != p.y) fp = p.y;
    const float all = fs + fp, inv = all == 0.f ? 0.f : 1.f / all;
    fs *= inv, fp *= inv;
#pragma unroll 1
    for (int e = 4 * lane; e < a.D; e += 4 * lanes) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (fs != 0.f) {
        const float4 x = *reinterpret_cast<const float4*>(a.own_o + row * a.D + e);
        o.x = fs * x.x, o.y = fs * x.y, o.z = fs * x.z, o.w = fs * x.w;
      }
      if (fp != 0.f) {
        const float4 x = *reinterpret_cast<const float4*>(a.pre_o + row * a.D + e);
        o.x = fmaf(fp, x.x, o.x), o.y = fmaf(fp, x.y, o.y), o.z = fmaf(fp, x.z, o.z), o.w = fmaf(fp, x.w, o.w);
      }
      *reinterpret_cast<uint2*>(a.out + row * a.D + e) = make_uint2(f32_to_bf16x2(o.x, o.y), f32_to_bf16x2(o.z, o.w));
    }
  }
}

size_t up(size_t n) { return (n + 1023) / 1024 * 1024; }

// the workspace: what the passes use (counters first), then the partial results of both
struct SharedLayout {
  size_t own_o, own_ml, pre_o, pre_ml, total;
};
SharedLayout layout(int T, int Hq, int Hkv, int D) {
  const size_t rows = (size_t)T * Hq;
  SharedLayout l;
  l.own_o = up(attn_kv8_workspace_size(Hq, Hkv, D));
  l.own_ml = l.own_o + up(rows * D * 4);
  l.pre_o = l.own_ml + up(rows * 8);
  l.pre_ml = l.pre_o + up(rows * D * 4);
  l.total = l.pre_ml + up(rows * 8);
  return l;
}

}  // namespace

size_t attn_kv8_shared_workspace_size(int T, int Hq, int Hkv, int D) { return layout(T, Hq, Hkv, D).total; }

cudaError_t launch_attn_kv8_shared(const AttnArgs& own, const AttnArgs& pre, int format, cudaStream_t stream, bool pdl) {
  const SharedLayout l = layout(own.T, own.Hq, own.Hkv, own.D);
  uint8_t* ws = static_cast<uint8_t*>(own.ws);
  AttnArgs s = own, p = pre;
  s.part_o = reinterpret_cast<float*>(ws + l.own_o), s.part_ml = reinterpret_cast<float2*>(ws + l.own_ml);
  p.part_o = reinterpret_cast<float*>(ws + l.pre_o), p.part_ml = reinterpret_cast<float2*>(ws + l.pre_ml);
  for (const AttnArgs* a : {&s, &p}) {
    const cudaError_t e = format == QG_KV_I8 ? launch_by_shape<QG_KV_I8, true>(*a, stream, pdl)
                                             : launch_by_shape<QG_KV_E4M3, true>(*a, stream, pdl);
    if (e != cudaSuccess) return e;
  }
  const JoinArgs j = {own.cu_q, pre.cu_req, own.R, pre.R, own.T, own.Hq, own.D, s.part_o, p.part_o, s.part_ml,
                      p.part_ml, own.out};
  const long long rows = (long long)own.T * own.Hq, per = kJoinThreads / 8;
  const int grid = (int)std::min<long long>((rows + per - 1) / per, 8LL * device_sm_count());
  return launch_kernel(attn_shared_join_kernel, dim3(grid), dim3(kJoinThreads), 0, stream, pdl, j);
}

}  // namespace qg
