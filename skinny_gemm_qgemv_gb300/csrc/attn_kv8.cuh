// What the two tensor-core kernels of attention over the 8-bit cache share: how
// a batch is cut into shares, and the conversions of codes.
#pragma once

#include <cstdint>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {

constexpr int kUnit = 16;                       // tokens that lie in one block, whatever its size: one scale pair
constexpr float kNoMax = -3.402823466e+38f;     // running maximum before any seen token: no finite score is below it
constexpr float kSlack = 8.f;                   // log2: probabilities stay below 2^8 (fp16 holds 2^15)
constexpr float kMinScale = 5.4210109e-20f;     // 2^-64
constexpr size_t kAttnCounterBytes = 4096;      // one counter per CTA
constexpr int kMaxCtas = 160;                   // CTAs, and so pieces of an item: their factors fit the combine buffer

constexpr int kMmaRows = 16;                    // query rows of an item of the warp-level kernel, at most
constexpr int kTcRows = 64;                     // query rows of an item of the tcgen05 kernel
constexpr int kTcHead = 128;                    // elements that it fills every head up to

// bytes of the partial results of one CTA's piece: fp32 outputs, then (max, sum) per row
__host__ __device__ constexpr size_t attn_piece_bytes(int rows, int D) { return (size_t)rows * (D * 4 + 8); }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t hsub2_1152(uint32_t a) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x64806480u));
  return r;
}
// codes (b0, b1) and (b2, b3) of a word as f16 pairs, exact. int8: b ^ 0x80 =
// b + 128 under the exponent byte 0x64 is fp16 1024 + 128 + b.
// (1152 comes off here and not off a product's sum: there it saves up to 3 %, 32 requests of four drafts 65.5 -> 63.5 us,
// but sums of codes near 0 then run through values a thousand times their own and lose as many bits.)
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == QG_KV_I8) {
    const uint32_t u = w ^ 0x80808080u;
    lo = prmt(u, 0x64646464u, 0x4140u);
    hi = prmt(u, 0x64646464u, 0x4342u);
    lo = hsub2_1152(lo), hi = hsub2_1152(hi);
  } else {
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The CTA's view of the batch: requests, their steps and where a step lies.
// A request has one item per key/value head and tile of kRows query rows, an
// item has ceil(tokens / tokens of a step) steps. Shares are cut on a scale on which an
// item also costs some steps before its first one: what beginning and ending it
// takes (a batch of 32 requests of 1..8192 tokens, where one CTA can
// meet 20 short items: 82 -> 60 us).
struct AttnBatch {
  const int* first;  // [R + 1] steps before the request
  const int* cost;   // [R + 1] the same with every item's cost
  const int* ctx;    // [R]
  const int* cu;     // [R + 1]
  int R, G;
};
struct AttnPlace {
  int r, h, rt;   // request, key/value head, row tile
  int s, steps;   // step within its item, steps of the item
};
// How a kernel cuts its items: tokens of a step, steps that an item costs before
// its first one, and up to how many steps an item is not cut at all.
template <int TOK, int COST, int WHOLE>
struct AttnCut {
  static constexpr int kTok = TOK, kCost = COST, kWhole = WHOLE;
};
template <int TOK>  // tokens of a step
__device__ __forceinline__ int attn_steps(int ctx) {
  return max(1, (ctx + TOK - 1) / TOK);
}
// largest r in [0, n) with v[r] <= x
__device__ __forceinline__ int attn_find(const int* v, int n, int x) {
  int lo = 0, hi = n;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
template <int ROWS, class CUT>
__device__ __forceinline__ AttnPlace attn_locate(const AttnBatch& b, int step) {
  AttnPlace p;
  p.r = attn_find(b.first, b.R, step);
  p.steps = attn_steps<CUT::kTok>(b.ctx[p.r]);
  const int tiles = ((b.cu[p.r + 1] - b.cu[p.r]) * b.G + ROWS - 1) / ROWS;
  const int rem = step - b.first[p.r], item = rem / p.steps;
  p.s = rem - item * p.steps;
  p.h = item / tiles;
  p.rt = item - p.h * tiles;
  return p;
}
// first step at or after place x of the cost scale, and the place of a step
template <class CUT>
__device__ __forceinline__ int attn_step_at(const AttnBatch& b, int x) {
  if (x >= b.cost[b.R]) return b.first[b.R];
  const int r = attn_find(b.cost, b.R, x), steps = attn_steps<CUT::kTok>(b.ctx[r]);
  const int rem = x - b.cost[r], item = rem / (steps + CUT::kCost), at = rem - item * (steps + CUT::kCost);
  // a short item belongs to the CTA whose share holds its beginning
  return b.first[r] + item * steps + (steps <= CUT::kWhole ? (at ? steps : 0) : max(0, at - CUT::kCost));
}
template <class CUT>
__device__ __forceinline__ int attn_cost_of(const AttnBatch& b, int step) {
  const int r = attn_find(b.first, b.R, step), steps = attn_steps<CUT::kTok>(b.ctx[r]);
  const int rem = step - b.first[r], item = rem / steps;
  return b.cost[r] + rem + (item + 1) * CUT::kCost;
}

// The batch's tables in shared memory, formed by all NT threads of a CTA (`part`
// has NT / 32 entries); returns the batch. The host has checked that the sums
// stay below 2^31 for query tokens that ascend within T; if they do not, the
// batch's cost is -1.
template <int ROWS, class CUT, int NT>
__device__ __forceinline__ AttnBatch attn_scan(const AttnArgs& a, int* first, int* cost, int* cus, int* ctxs,
                                               int2* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.Hq / a.Hkv;
  const int per = (a.R + NT - 1) / NT;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  const int most = a.max_blocks * a.bs;
  int2 mine = make_int2(0, 0);
  bool bad = false;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const int q0 = a.cu_q[r], q1 = a.cu_q[r + 1];
    bad |= q0 < 0 || q0 > q1 || q1 > a.T;
    int ctx = max(0, a.ctx_lens[r]);
    if (ctx > most) {
      ctx = most;
      if (blockIdx.x == 0) report_error(a.err, kErrKvLength);
    }
    ctxs[r] = ctx;
    cus[r] = q0;
    if (r == a.R - 1) cus[a.R] = q1;
    first[r] = mine.x;
    cost[r] = mine.y;
    const int items = a.Hkv * (((q1 - q0) * G + ROWS - 1) / ROWS), steps = attn_steps<CUT::kTok>(ctx);
    mine.x += items * steps;
    mine.y += items * (steps + CUT::kCost);
  }
  int2 inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) inc.x += x, inc.y += y;
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 31) part[warp] = make_int2(inc.x, bad ? -1 : inc.y);
  __syncthreads();
  int2 before = make_int2(inc.x - mine.x, inc.y - mine.y), total = make_int2(0, 0);
  int marks = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int2 x = part[w];
    if (w < warp) before.x += x.x, before.y += x.y;
    total.x += x.x, total.y += x.y;
    marks |= x.y;
  }
#pragma unroll 1
  for (int r = r0; r < r1; ++r) first[r] += before.x, cost[r] += before.y;
  if (threadIdx.x == 0) first[a.R] = total.x, cost[a.R] = marks < 0 ? -1 : total.y;
  __syncthreads();
  return {first, cost, ctxs, cus, a.R, G};
}

// This CTA's share of the batch: steps c0 .. c1 - 1 (none if c0 == c1).
struct AttnShare {
  int c0, c1, share, more;
};
template <class CUT>
__device__ __forceinline__ AttnShare attn_share(const AttnBatch& b, uint32_t* err) {
  const int W = b.cost[b.R], A = min((int)gridDim.x, W);  // the first W % A CTAs take one place more than the others
  AttnShare s = {0, 0, 0, 0};
  if ((int)blockIdx.x >= A) {
    if (W < 0 && blockIdx.x == 0 && threadIdx.x == 0) report_error(err, kErrKvQueries);
    return s;
  }
  s.share = W / A, s.more = W % A;
  // both ends side by side, by the even and the odd lanes
  const int i = blockIdx.x + (threadIdx.x & 1), step = attn_step_at<CUT>(b, i * s.share + min(i, s.more));
  s.c0 = __shfl_sync(0xffffffffu, step, 0);
  s.c1 = __shfl_sync(0xffffffffu, step, 1);
  return s;
}
// the CTA whose share holds a step
template <class CUT>
__device__ __forceinline__ int attn_cta_of(const AttnBatch& b, const AttnShare& s, int step) {
  const int x = attn_cost_of<CUT>(b, step), big = s.more * (s.share + 1);
  return x < big ? x / (s.share + 1) : s.more + (x - big) / s.share;
}

}  // namespace qg
