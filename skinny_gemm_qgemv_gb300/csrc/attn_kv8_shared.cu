// Attention of requests whose groups share a prefix of the paged 8-bit cache.
//
// With z_j the scores of a row, the sums over the shared prefix P and over the
// request's own tokens S join as
//   m = max(m_P, m_S), out = (2^(m_P - m) l_P o_P + 2^(m_S - m) l_S o_S) /
//                            (2^(m_P - m) l_P + 2^(m_S - m) l_S),
// so the prefix is read for all query rows of its group together instead of once
// per request. Three launches: every request over its own tokens, every group over its
// prefix (no mask: all of it is seen), both leaving a row's maximum, sum and fp32
// output in the workspace, and the joining.
//
// Measured (32/8 heads of 128): four requests of up to 37 own tokens over 600 shared ones 19 us, 34 of up to 1024 over
// 8200 43 us, 64 of up to 300 over 65529 106 us, of which the own tokens' pass takes 14 to 22
// and the joining 6 to 8; the prefix's kernel begins while the own tokens' one ends. The own tokens always go to the
// warp-level kernel, a pass per 16 rows: more rows a request over many own tokens take longer than by attn_kv8_paged, whose
// tcgen05 kernel leaves no partial results (64 requests of eight drafts, 8 heads a group, up to 1000 own tokens over 8192
// shared ones 319 us; attn_kv8_paged over the own tokens alone 71).
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_kv8_mma.cuh"
#include "attn_prefix.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

struct JoinArgs {
  const int32_t *cu_q, *cu_req;
  int R, groups, T, Hq, D;
  const float *own_o, *pre_o;
  const float2 *own_ml, *pre_ml;
  const int2* source;     // null: every row's prefix result is in pre_o
  const uint8_t* pieces;
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

// Two rows a CTA, four warps a row. What a row consists of: the request's own tokens; where its group has a prefix, that
// one's result or, if the prefix's steps went over several CTAs, their pieces, every fourth one a warp's (one warp a row
// took 10 us for 1088 rows of 19 pieces, 6 us with four). The order of the sums depends on shapes and lengths alone.
__global__ void __launch_bounds__(kJoinThreads) attn_shared_join_kernel(JoinArgs a) {
  __shared__ float4 sums[kJoinThreads / 32][32];
  pdl_wait();
  pdl_launch_dependents();
  const bool bad = bounds_bad(a.cu_q, a.R, a.T);
  if (bounds_bad(a.cu_req, a.groups, a.R) || bad) return;
  const int r0 = a.cu_q[0] * a.Hq, r1 = a.cu_q[a.R] * a.Hq;
  const int g0 = a.cu_q[a.cu_req[0]] * a.Hq, g1 = a.cu_q[a.cu_req[a.groups]] * a.Hq;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & 3;
  // (a sum that is no number makes the row none, as it would alone)
  auto weight = [&](float2 s, float m) { return s.y > 0.f ? s.y * ex2(s.x - m) : s.y; };
#pragma unroll 1
  for (int pair = r0 + 2 * blockIdx.x; pair < r1; pair += 2 * gridDim.x) {
    const int row = pair + (warp >> 2);
    const bool live = row < r1, shared = live && row >= g0 && row < g1;
    const float2 none = make_float2(kNoMax, 0.f);
    float2 own = none, pre = none;
    int2 from = make_int2(0, shared ? 1 : 0);
    if (live) own = a.own_ml[row];
    if (shared) {
      if (a.source) from = a.source[row];
      pre = a.pre_ml[row];  // (not written where the prefix is in pieces)
    }
    const int pieces = from.y;
    // the first piece is the second one of its CTA, as its item goes on after it; the others begin theirs
    auto piece = [&](int p) {
      return a.pieces + (size_t)(2 * ((from.x >> 8) + p) + (p == 0 ? 1 : 0)) * prefix_piece_bytes(a.D);
    };
    auto stat = [&](int p) {
      return p >= pieces ? none : pieces == 1 ? pre
                                              : reinterpret_cast<const float2*>(piece(p) + (size_t)kPrefixRows * a.D * 4)[from.x & 255];
    };
    float2 mine = stat(lane);  // of piece `lane`; further ones are read again
    float m = fmaxf(own.x, mine.x);
#pragma unroll 1
    for (int p = lane + 32; p < pieces; p += 32) m = fmaxf(m, stat(p).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float all = weight(mine, m) + (lane == 0 ? weight(own, m) : 0.f);
#pragma unroll 1
    for (int p = lane + 32; p < pieces; p += 32) all += weight(stat(p), m);
    all = warp_sum(all);
    const float inv = all == 0.f ? 0.f : 1.f / all;
#pragma unroll 1
    for (int e0 = 0; e0 < a.D; e0 += 128) {
      const int e = e0 + 4 * lane;
      const bool in = e < a.D;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](float w, const float* src) {
        if (in && w != 0.f) {
          const float4 x = *reinterpret_cast<const float4*>(src + e);
          o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y), o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
        }
      };
      if (part == 0) add(weight(own, m) * inv, a.own_o + (size_t)row * a.D);
      if (part == 1 && pieces == 1) add(weight(pre, m) * inv, a.pre_o + (size_t)row * a.D);
      if (pieces > 1) {
#pragma unroll 1
        for (int p0 = 0; p0 < pieces; p0 += 32) {
          const float w = weight(p0 ? stat(p0 + lane) : mine, m) * inv;
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float wk = __shfl_sync(0xffffffffu, w, k + part);  // (0 past the last piece)
            add(wk, reinterpret_cast<const float*>(piece(p0 + k + part)) + (size_t)(from.x & 255) * a.D);
          }
        }
      }
      sums[warp][lane] = o;
      __syncthreads();
      if (part == 0 && live && in) {
#pragma unroll
        for (int k = 1; k < 4; ++k) {
          const float4 x = sums[warp + k][lane];
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
        *reinterpret_cast<uint2*>(a.out + (size_t)row * a.D + e) =
            make_uint2(f32_to_bf16x2(o.x, o.y), f32_to_bf16x2(o.z, o.w));
      }
      __syncthreads();
    }
  }
}

size_t up(size_t n) { return (n + 1023) / 1024 * 1024; }

// the workspace: what the passes use (counters first), then the partial results of both
struct SharedLayout {
  size_t own_o, own_ml, pre_o, pre_ml, source, pieces, total;
};
// heads that attn_kv8_prefix.cu takes; its CTAs
bool prefix_tc_ok(int D) { return D <= 128; }
int prefix_ctas() { return device_sm_count(); }
SharedLayout layout(int T, int Hq, int Hkv, int D) {
  const size_t rows = (size_t)T * Hq;
  SharedLayout l;
  l.own_o = up(attn_kv8_workspace_size(Hq, Hkv, D));
  l.own_ml = l.own_o + up(rows * D * 4);
  l.pre_o = l.own_ml + up(rows * 8);
  l.pre_ml = l.pre_o + up(rows * D * 4);
  l.source = l.pre_ml + up(rows * 8);
  l.pieces = l.source + (prefix_tc_ok(D) ? up(rows * 8) : 0);
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
  // Up to 16 rows a group, on the average of the batch (the groups' own rows are known to the GPU alone; a group of 64 beside
  // 19 of one, two heads a group, goes to the warp-level kernel with the others), of a prefix that may be long, the warp-level kernel reads it at the copy rate, where that of
  // attn_kv8_prefix.cu takes as long for 128 rows as for one. Measured, here and there (32/8 heads of 128): 16 rows, 600
  // tokens 20.0 and 21.9 us, 4096 tokens 27.1 and 23.5, 65536 tokens 65 and 51; 32 rows, 65536 tokens 68 and 71, 64 rows 69
  // and 113.
  const bool tc = prefix_tc_ok(own.D) && !(attn_rows(pre) <= 16 && (long long)pre.max_blocks * pre.bs >= 2048);
  auto warp_level = [&](const AttnArgs& a) {
    return format == QG_KV_I8 ? launch_by_shape<QG_KV_I8, true>(a, stream, pdl)
                              : launch_by_shape<QG_KV_E4M3, true>(a, stream, pdl);
  };
  cudaError_t e = warp_level(s);
  if (e != cudaSuccess) return e;
  int2* source = tc ? reinterpret_cast<int2*>(ws + l.source) : nullptr;
  e = tc ? launch_attn_kv8_prefix(p, format, ws + l.pieces, source, prefix_ctas(), stream, pdl) : warp_level(p);
  if (e != cudaSuccess) return e;
  const JoinArgs j = {own.cu_q, pre.cu_req, own.R, pre.R, own.T, own.Hq, own.D, s.part_o, p.part_o, s.part_ml, p.part_ml,
                      source, ws + l.pieces, own.out};
  const long long rows = (long long)own.T * own.Hq, per = 2;
  const int grid = (int)std::min<long long>((rows + per - 1) / per, 8LL * device_sm_count());
  return launch_kernel(attn_shared_join_kernel, dim3(grid), dim3(kJoinThreads), 0, stream, pdl, j);
}

}  // namespace qg
