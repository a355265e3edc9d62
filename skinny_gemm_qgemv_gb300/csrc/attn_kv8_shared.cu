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
#include "attn_prefix.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

struct JoinArgs {
  AttnArgs own, pre;
  const uint8_t* pieces;  // null: the prefix pass leaves every row's result in pre.part_o
  int ctas;               // of the prefix pass
};

constexpr int kJoinThreads = 256;

// true in all threads where the bounds do not ascend within T (the passes have reported it and computed nothing)
__device__ bool bounds_bad(const int32_t* cu, int n, int top) {
  bool bad = false;
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= cu[i] < 0 || cu[i] > cu[i + 1] || cu[i + 1] > top;
  return __syncthreads_or(bad);
}

// A row per warp. Its parts: the request's own tokens; where its group has a prefix, that one's result or, if the
// prefix's steps went over several CTAs, their pieces, in the order of the CTAs.
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(const __grid_constant__ JoinArgs j) {
  extern __shared__ int tables[];
  __shared__ int2 scan_part[kJoinThreads / 32];
  const AttnArgs& a = j.own;
  pdl_wait();
  pdl_launch_dependents();
  if (bounds_bad(a.cu_q, a.R, a.T) || bounds_bad(j.pre.cu_req, j.pre.R, a.R)) return;
  const int t0 = a.cu_q[0], t1 = a.cu_q[a.R], G = a.Hq / a.Hkv, groups = j.pre.R;
  AttnBatch batch = {};
  int *first = tables, *cost = first + groups + 1, *cus = cost + groups + 1, *ctxs = cus + groups + 1;
  AttnShare share = {0, 0, 0, 0};
  if (j.pieces) {
    batch = attn_scan<kPrefixRows, PrefixCut, kJoinThreads, true>(j.pre, first, cost, cus, ctxs, scan_part);
    const int W = cost[groups], A = min(j.ctas, W);  // as attn_share
    if (A > 0) share.share = W / A, share.more = W % A;
  }
  const int g0 = a.cu_q[j.pre.cu_req[0]], g1 = a.cu_q[j.pre.cu_req[groups]];
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)(t1 - t0) * a.Hq;
#pragma unroll 1
  for (long long i = (long long)blockIdx.x * (kJoinThreads / 32) + threadIdx.x / 32; i < rows;
       i += (long long)gridDim.x * (kJoinThreads / 32)) {
    const int t = t0 + (int)(i / a.Hq), hq = (int)(i % a.Hq);
    const long long row = (long long)t0 * a.Hq + i;
    const float2 own = a.part_ml[row];
    const bool shared = t >= g0 && t < g1;
    int f = 0, pieces = shared ? 1 : 0, rr = 0;
    const float* pre_o = j.pre.part_o + row * a.D;
    const float2* pre_ml = j.pre.part_ml + row;
    if (shared && j.pieces) {
      const int g = attn_find(cus, groups, t);  // the last group that begins here: one with query tokens
      const int rho = (t - cus[g]) * G + hq % G, tiles = ((cus[g + 1] - cus[g]) * G + kPrefixRows - 1) / kPrefixRows;
      const int steps = attn_steps<kPrefixTok>(ctxs[g]), at = first[g] + ((hq / G) * tiles + rho / kPrefixRows) * steps;
      f = attn_cta_of<PrefixCut>(batch, share, at);
      pieces = attn_cta_of<PrefixCut>(batch, share, at + steps - 1) - f + 1;
      rr = rho % kPrefixRows;
    }
    // the first piece is the second one of its CTA, as its item goes on after it; the others begin theirs
    auto piece = [&](int p) { return j.pieces + (size_t)(2 * (f + p) + (p == 0 ? 1 : 0)) * prefix_piece_bytes(a.D); };
    auto stat = [&](int p) {
      return pieces == 1 ? *pre_ml : reinterpret_cast<const float2*>(piece(p) + (size_t)kPrefixRows * a.D * 4)[rr];
    };
    // (a sum that is no number makes the row none, as it would alone)
    auto weight = [&](float2 s, float m) { return s.y > 0.f ? s.y * ex2(s.x - m) : s.y; };
    float m = own.x, all;
    for (int p = lane; p < pieces; p += 32) m = fmaxf(m, stat(p).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    all = lane == 0 ? weight(own, m) : 0.f;
    for (int p = lane; p < pieces; p += 32) all += weight(stat(p), m);
    all = warp_sum(all);
    const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll 1
    for (int e = 4 * lane; e < (a.D + 127) / 128 * 128; e += 128) {
      const bool in = e < a.D;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float w, const float* src) {
        if (in && w != 0.f) {
          const float4 x = *reinterpret_cast<const float4*>(src + e);
          o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y), o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
        }
      };
      add(weight(own, m) * inv, a.part_o + row * a.D);
      if (pieces == 1) {
        add(weight(*pre_ml, m) * inv, pre_o);
      } else {
#pragma unroll 4
        for (int p = 0; p < pieces; ++p)
          add(weight(stat(p), m) * inv, reinterpret_cast<const float*>(piece(p)) + (size_t)rr * a.D);
      }
      if (in)
        *reinterpret_cast<uint2*>(a.out + row * a.D + e) = make_uint2(f32_to_bf16x2(o.x, o.y), f32_to_bf16x2(o.z, o.w));
    }
  }
}

size_t up(size_t n) { return (n + 1023) / 1024 * 1024; }

// the workspace: what the passes use (counters first), then the partial results of both
struct SharedLayout {
  size_t own_o, own_ml, pre_o, pre_ml, pieces, total;
};
// the prefix pass by attn_kv8_prefix.cu; its CTAs
bool prefix_tc_ok(int D) { return D <= 128; }
int prefix_ctas() { return device_sm_count(); }
SharedLayout layout(int T, int Hq, int Hkv, int D) {
  const size_t rows = (size_t)T * Hq;
  SharedLayout l;
  l.own_o = up(attn_kv8_workspace_size(Hq, Hkv, D));
  l.own_ml = l.own_o + up(rows * D * 4);
  l.pre_o = l.own_ml + up(rows * 8);
  l.pre_ml = l.pre_o + up(rows * D * 4);
  l.pieces = l.pre_ml + up(rows * 8);
  l.total = l.pieces + (prefix_tc_ok(D) ? up(2 * prefix_ctas() * prefix_piece_bytes(D)) : 0);
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
  const bool tc = prefix_tc_ok(own.D);
  auto warp_level = [&](const AttnArgs& a) {
    return format == QG_KV_I8 ? launch_by_shape<QG_KV_I8, true>(a, stream, pdl)
                              : launch_by_shape<QG_KV_E4M3, true>(a, stream, pdl);
  };
  cudaError_t e = warp_level(s);
  if (e != cudaSuccess) return e;
  e = tc ? launch_attn_kv8_prefix(p, format, ws + l.pieces, prefix_ctas(), stream, pdl) : warp_level(p);
  if (e != cudaSuccess) return e;
  const JoinArgs j = {s, p, tc ? ws + l.pieces : nullptr, prefix_ctas()};
  const long long rows = (long long)own.T * own.Hq, per = kJoinThreads / 32;
  const int grid = (int)std::min<long long>((rows + per - 1) / per, 8LL * device_sm_count());
  return launch_kernel(attn_shared_join_kernel, dim3(grid), dim3(kJoinThreads), 16 * ((size_t)pre.R + 1), stream, pdl, j);
}

}  // namespace qg
