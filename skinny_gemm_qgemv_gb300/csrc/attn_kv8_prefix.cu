// Attention of the query rows of whole groups over their shared prefixes in the
// paged 8-bit cache, heads of up to 128 elements, on the 5th-generation tensor cores.
//
//   S [128 rows][128 tokens] = q K^T   A = the queries, B = the keys, both fp16 in
//                                      shared memory (codes and queries are exact)
//   P = 2^(S ks f + log2 vs - m)       a thread per query row: f the row's scale,
//                                      ks, vs the scales of the token's block
//   O [128 rows][D] += P V             A = P as fp16 in tensor memory, over the S that
//                                      it came from; B = the values, token-major
// There is no mask but the prefix's end: a step's tokens are seen by all rows, so
// rows stand across a CTA's lanes (S^T, as in attn_kv8_tc.cu, would need a vote
// on maxima across threads). m moves only where a score outgrows it by 2^8.
//
// An item is up to 256 rows of a key/value head; its steps go through two streams of
// MMAs and softmax warps that take turns on the tensor cores. With more than 128
// rows a stream is half of the rows, and both use a step's converted keys and
// values; with fewer the streams take every other step for the same rows and are
// added up at the end (one stream alone would wait for its own softmax half of the
// time).
//
// Warps: 0-3 and 4-7 softmax of the streams, 8-11 copy and convert keys, 12-15
// values, 16 looks up blocks and scales, 17 issues the MMAs. Codes go from global memory through
// registers to fp16 tiles: staged by TMA they would cross shared memory twice more
// (64 of 320 KB a step, whose 128 bytes a cycle the MMAs' operands need).
//
// Measured (32/8 heads of 128, int8): 64 requests over 65529 shared tokens, own tokens and join included, 106 us (16.8
// million scores a key/value head: 36 us at the library product's rate, 23 us for the bytes). A step of 256 rows and
// 128 tokens takes some 4100 cycles: each stream's chain of scores from tensor memory, exponentials and P back to it
// takes 2000, the MMAs of both 2900 in the tensor pipe's one order; it is busy for 24 % of a short run's cycles and the
// softmax warps issue in 39 %. With up to 128 rows a step takes 2500. Beginning and end cost 15 us: first codes, blocks'
// places and queries 6, results 3, the rest launch.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_kv8.cuh"
#include "attn_prefix.cuh"
#include "attn_tc.cuh"
#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 640;  // five warpgroups, the last with two warps at work
constexpr int kSlots = 8;       // steps whose blocks and scales are kept
constexpr int kRowsTile = 128;  // rows of a stream's MMAs
constexpr int kUnits = kPrefixTok / kUnit;
constexpr int TOK = kPrefixTok;

// DP: elements that a head is filled up to (64 or 128)
template <int DP>
struct PrefixShape {
  static constexpr int kHalves = DP / 64;            // 64-element blocks of a tile's rows
  static constexpr int kTile = TOK * DP * 2;         // 128 rows (tokens or queries) as fp16
  static constexpr int kBlock = TOK * 128;           // one 64-element block of them
  static constexpr int kTokens = 32 / kHalves;       // tokens of a load of all converters
  static constexpr int kLoads = TOK / kTokens;
  static constexpr int kSmem = 6 * kTile;            // two of queries, keys and values each
  static constexpr uint32_t kColS = 0, kColO = 256;  // tensor memory columns: S0, S1, O0, O1, 128 apart
};

__device__ __forceinline__ void tmem_ld32(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t));
}
// two waits' worth of operands: orders later uses of v[0..31] after the loads
__device__ __forceinline__ void tmem_wait_ld32(float* v) {
  tmem_wait_ld(v);
  tmem_wait_ld(v + 16);
}
constexpr float kMostMass = 256.f;  // sum of some p up to which their maximum stays: fp16 holds 2^15

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 bytes of global memory, zeros where `there` is not set; no branch
__device__ __forceinline__ uint4 load_if(const void* p, bool there) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((unsigned)there)
      : "memory");
  return v;
}

// A warpgroup's share of the registers that the CTA was launched with: 96 a thread, of which the softmax gets more
// (256 x 128 + 384 x 72 <= 640 x 96).
constexpr int kSoftmaxRegs = 128, kOtherRegs = 72;
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int FMT, int DP>
__global__ void __launch_bounds__(kThreads, 1) attn_kv8_prefix_kernel(AttnArgs a, uint8_t* pieces, int2* source) {
  using S = PrefixShape<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = warp & 3;
  uint8_t* qbuf = smem;
  uint8_t* kbuf = qbuf + 2 * S::kTile;
  uint8_t* vbuf = kbuf + 2 * S::kTile;
  int* first = reinterpret_cast<int*>(vbuf + 2 * S::kTile);
  int* cost = first + a.R + 1;
  int* cus = cost + a.R + 1;
  int* ctxs = cus + a.R + 1;
  __shared__ long long unit_at[kSlots][kUnits];     // element of the unit's first token in the cache, -1: not there
  __shared__ bool plain[kSlots];                    // all of the slot's units are of kind 1
  __shared__ float4 unit_scales[kSlots][kUnits];    // key scale, log2 of the value scale, 2^-that, kind
  // a step's blocks, its scales have been written; its values have been multiplied
  __shared__ uint64_t found[kSlots], scaled[kSlots], spent[kSlots];
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], s_full[2], p_ready[2], q_full, o_done;
  __shared__ int2 scan_part[kThreads / 32];
  __shared__ float2 other[kRowsTile];  // the second stream's maxima and sums
  __shared__ uint32_t tmem_base;
  __shared__ volatile uint32_t abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(found + i, 1), mbar_init(scaled + i, 1), mbar_init(spent + i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4), mbar_init(v_full + i, 4);
      mbar_init(k_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + i, 4);
    }
    mbar_init(&q_full, 8);
    mbar_init(&o_done, 1);
    abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 17) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // The kernel before is the one over the requests' own tokens, of whose results nothing is read here: its CTAs all
  // waited for what came before them (the cache, the lengths, the last call's joining) before they let this one begin, so
  // it need not wait for it but at its end, before the joining begins. What is read below was complete by then; the fence
  // keeps loads from what an SM's L1 may hold of older contents.
  __threadfence();
  pdl_launch_dependents();
  tc_before();
  const AttnBatch batch = attn_scan<kPrefixRows, PrefixCut, kThreads, true>(a, first, cost, cus, ctxs, scan_part);
  tc_after();
  const AttnShare share = attn_share<PrefixCut>(batch, a.err);
  const uint32_t tbase = tmem_base;

  // by a whole warp, which goes on together
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    // (in line: around a call ptxas finds no registers for setmaxnreg's shares)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = false;
#pragma unroll 1
    for (uint32_t i = 0; i < kMaxPolls && !ok; ++i) {
      ok = mbar_try_wait(bar, parity);
      if (!ok && abort_flag) break;
      if (!ok && i == kMaxPolls - 1) {
        report_error(a.err, kErrAttnWait);
        abort_flag = 1u;
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  // A segment: the steps of one item in this CTA's share. Every role walks the segments by itself; the steps of the CTA
  // are counted through (step g: buffers g & 1, slot g % kSlots).
  struct Segment {
    AttnPlace item;
    int n, g, rows, tok0, index;
  };
  auto first_segment = [&]() {
    Segment s;
    s.n = s.g = 0;
    s.index = -1;
    return s;
  };
  auto next_segment = [&](Segment& s, int& step) {
    step += s.n;
    if (step >= share.c1) return false;
    s.g += s.n;
    ++s.index;
    s.item = attn_locate<kPrefixRows, PrefixCut>(batch, step);
    s.n = min(share.c1, step - s.item.s + s.item.steps) - step;
    s.rows = min(kPrefixRows, (cus[s.item.r + 1] - cus[s.item.r]) * batch.G - s.item.rt * kPrefixRows);
    s.tok0 = s.item.s * TOK;
    return true;
  };
  int step = share.c0;
  Segment sg = first_segment();

  if (warp < 8) {
    registers_up<kSoftmaxRegs>();
    // ------------------------------------------------ softmax: a row per thread
    const int stream = warp >> 2, r = quad * 32 + lane;
    const uint32_t tlane = tbase + ((uint32_t)(quad * 32) << 16);
    const uint32_t ts = tlane + S::kColS + 128 * stream, to = tlane + S::kColO + 128 * stream;
    uint32_t passes = 0;  // of s_full[stream]
    while (next_segment(sg, step)) {
      const bool two = sg.rows > kRowsTile;
      const int ctx = ctxs[sg.item.r], q0 = cus[sg.item.r];
      const int rr = (two ? kRowsTile * stream : 0) + r;
      const int rho = sg.item.rt * kPrefixRows + rr, qi = rho / batch.G;
      const bool live = rr < sg.rows;
      const size_t out_row = (size_t)(q0 + qi) * a.Hq + sg.item.h * batch.G + rho - qi * batch.G;
      // the row as 2^-sigma q in fp16, exact, sigma from its largest finite element
      float rf;
      {
        // copied as they are to their place, a warp's 32 rows by that warp, then converted there
        const long long at = (long long)(q0 + qi) * a.q_stride + (long long)(sg.item.h * batch.G + rho - qi * batch.G) * a.D;
        const uint32_t rows = smem_u32(qbuf) + stream * S::kTile + quad * 32 * 128;
        auto chunk = [&](int row, int j) { return rows + (j >> 3) * S::kBlock + row * 128 + (((j & 7) ^ (row & 7)) << 4); };
        constexpr int kLanes = DP / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows of a copy
#pragma unroll 4
        for (int i = 0; i < kLanes; ++i) {
          const int k = i * kAtOnce + lane / kLanes, j = lane % kLanes;
          const long long from = __shfl_sync(0xffffffffu, live ? at : -1ll, k);
          cp_async16(chunk(k, j), a.q + (from < 0 ? 0 : from + 8 * j), from >= 0 && 8 * j < a.D);
        }
        cp_async_wait_all();
        __syncwarp();
        unsigned most = 0u;
#pragma unroll 4
        for (int j = 0; j < DP / 8; ++j) {
          const uint4 raw = lds128(chunk(lane, j));
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned lo = w[k] << 16 & 0x7FFF0000u, hi = w[k] & 0x7FFF0000u;
            most = max(most, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
          }
        }
        const int sigma = fp16_prescale_exp(__uint_as_float(most));
        const float down = pow2f(-sigma);
        rf = a.scale_log2 * pow2f(sigma);
#pragma unroll 4
        for (int j = 0; j < DP / 8; ++j) {
          const uint4 raw = lds128(chunk(lane, j));
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
          uint32_t f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            f[k] = f16x2(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xFFFF0000u) * down);
          sts128(chunk(lane, j), make_uint4(f[0], f[1], f[2], f[3]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
      float m = kNoMax, l = 0.f;
      bool begun = false, fresh = true, large = false;  // fresh: no maximum yet
#pragma unroll 1
      for (int i = two ? 0 : stream; i < sg.n; i += two ? 1 : 2) {
        const int g = sg.g + i, slot = g % kSlots;
        wait_warp(scaled + slot, g / kSlots & 1);
        wait_warp(s_full + stream, passes & 1);
        ++passes;
        tc_after();
        const int seen = ctx - (sg.tok0 + i * TOK);  // tokens of the step, if not all
        const float4* us = unit_scales[slot];
        // Two units (32 columns) at a time: p against the maximum so far, its sum without the value scale, and as fp16 over
        // the scores read before. Where the sum is at most 2^8 so is every p, and m stays (a pass over the scores for their
        // maximum took as long as the exponentials).
        int c = 0;
        if (!fresh && !large && plain[slot] && seen >= TOK) {
          // nothing to mask: the next scores are on the way while these are worked on
          float s[2][32];
          auto half = [&](float(&e)[32], int c) {
            const float4 sc[2] = {us[2 * c], us[2 * c + 1]};
            uint32_t p[16];
            float mass = 0.f, part = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint64_t f2 = both(sc[u].x * rf), b2 = both(sc[u].y - m);
              uint64_t sum = 0ull;
#pragma unroll
              for (int j = 16 * u; j < 16 * u + 16; j += 2) {
                float y0, y1;
                unpair2(ffma2(pair2(__float_as_uint(e[j]), __float_as_uint(e[j + 1])), f2, b2), y0, y1);
                y0 = ex2(y0), y1 = ex2(y1);
                sum = fadd2(sum, pair2(__float_as_uint(y0), __float_as_uint(y1)));
                p[j / 2] = f16x2(y0, y1);
              }
              float s0, s1;
              unpair2(sum, s0, s1);
              mass += s0 + s1;
              part = fmaf(s0 + s1, sc[u].z, part);
            }
            if (__any_sync(0xffffffffu, mass > kMostMass)) return false;
            l += part;
            tmem_st16(ts + 16 * c, *reinterpret_cast<float(*)[16]>(p));
            return true;
          };
          tmem_ld32(ts, s[0]);
#pragma unroll 1
          for (; c < TOK / 32; c += 2) {
            tmem_wait_ld32(s[0]);
            tmem_ld32(ts + 32 * c + 32, s[1]);
            const bool first = half(s[0], c);
            tmem_wait_ld32(s[1]);
            if (!first) break;
            if (c == 0) tmem_ld32(ts + 64, s[0]);
            if (!half(s[1], c + 1)) {
              ++c;
              break;
            }
          }
          tmem_wait_ld32(s[0]);
        }
        // The general form: m rises to a whole number above the largest score, by which what the step has written already
        // is scaled exactly.
#pragma unroll 1
        for (; c < TOK / 32; ++c) {
          const float4 sc[2] = {us[2 * c], us[2 * c + 1]};
          const int here = seen - 32 * c;
          const bool edge = here < 32 || sc[0].w == 0.f || sc[1].w == 0.f;
          uint32_t p[16];
          float s[32], part = 0.f;
          // (twice at most: above a whole number that no score passes there is no second rise)
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            tmem_ld32(ts + 32 * c, s);
            tmem_wait_ld32(s);
            if (!fresh) {
              float mass = 0.f;
              part = 0.f;
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint64_t f2 = both(sc[u].x * rf), b2 = both(large ? sc[u].y : sc[u].y - m), m2 = both(-m);
                uint64_t sum = 0ull;
                float* e = s + 16 * u;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  float y0, y1;
                  // (large scores: as they are compared with m, then the difference; in one step it may lie above 0 by their
                  // rounding)
                  uint64_t y = ffma2(pair2(__float_as_uint(e[j]), __float_as_uint(e[j + 1])), f2, b2);
                  if (large) y = fadd2(y, m2);
                  unpair2(y, y0, y1);
                  e[j] = ex2(y0), e[j + 1] = ex2(y1);
                }
                if (edge) {
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    if (sc[u].w == 0.f || 16 * u + j >= here) e[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                  sum = fadd2(sum, pair2(__float_as_uint(e[j]), __float_as_uint(e[j + 1])));
                  p[8 * u + j / 2] = f16x2(e[j], e[j + 1]);
                }
                float s0, s1;
                unpair2(sum, s0, s1);
                mass += s0 + s1;
                part = fmaf(s0 + s1, sc[u].z, part);
              }
              if (pass == 1 || !__any_sync(0xffffffffu, mass > kMostMass)) break;
              tmem_ld32(ts + 32 * c, s);
              tmem_wait_ld32(s);
            }
            fresh = false;
            float top = kNoMax;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float4 x = sc[j / 16];
              if (j < here && x.w != 0.f) top = fmaxf(top, fmaf(s[j], x.x * rf, x.y));
            }
            const float mn = top > m ? ceilf(top) : m, f = ex2(m - mn);
            const uint32_t f16 = f16x2(f, f);
            m = mn;
            large = __any_sync(0xffffffffu, fabsf(m) > 65536.f && m != kNoMax);
            l *= f;
#pragma unroll 1
            for (int k = 0; k < c; ++k) {
              uint32_t x[16];
              tmem_ld16(ts + 16 * k, reinterpret_cast<float*>(x));
              tmem_wait_ld(reinterpret_cast<float*>(x));
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] = hmul2(x[j], f16);
              tmem_st16(ts + 16 * k, *reinterpret_cast<float(*)[16]>(x));
            }
            if (begun) {  // (the stream's last product has been waited for with this S)
#pragma unroll 1
              for (int k = 0; k < DP / 16; ++k) {
                float o[16];
                tmem_ld16(to + 16 * k, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= f;
                tmem_st16(to + 16 * k, o);
              }
            }
          }
          l += part;
          if (sc[0].w == 2.f || sc[1].w == 2.f) {  // of a block of zero scale only the probabilities count
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (sc[j / 8].w == 2.f) p[j] = 0u;
          }
          tmem_st16(ts + 16 * c, *reinterpret_cast<float(*)[16]>(p));
        }
        begun = true;
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + stream);
      }
      // ---- the segment's results ----
      wait_warp(&o_done, sg.index & 1);
      tc_after();
      float w0 = 1.f, w1 = 0.f;  // weights of the streams' outputs
      if (!two) {
        if (stream == 1) other[r] = make_float2(m, l);
        named_barrier<256>(1);
        if (stream == 0) {
          const float2 x = other[r];
          const float mn = fmaxf(m, x.x);
          w0 = ex2(m - mn), w1 = ex2(x.x - mn);
          l = fmaf(x.y, w1, l * w0);
          m = mn;
        }
      }
      const float inv = l == 0.f ? 0.f : __frcp_rn(l);
      w0 *= inv, w1 *= inv;
      const bool second = !two && sg.n > 1;  // (the streams' outputs are sums from their first step on)
      if (two || stream == 0) {
        const int item_first = step - sg.item.s;
        const bool whole = item_first >= share.c0 && item_first + sg.item.steps <= share.c1;
        const int last = whole ? 0 : attn_cta_of<PrefixCut>(batch, share, item_first + sg.item.steps - 1);
        uint8_t* piece = prefix_piece(pieces, blockIdx.x, item_first < share.c0 ? 0 : 1, a.D);
        if (live) {
          float2* ml = whole ? a.part_ml + out_row : reinterpret_cast<float2*>(piece + (size_t)kPrefixRows * a.D * 4) + rr;
          *ml = make_float2(m, l);
          if (item_first >= share.c0)  // the CTA that has the item's beginning says how many pieces it is in
            source[out_row] = make_int2(blockIdx.x << 8 | rr, whole ? 1 : last - (int)blockIdx.x + 1);
        }
        // 32 rows and elements of a warp at a time through the queries' place (their products are done), so that a row's
        // 128 bytes are stored together
        const uint32_t stage = smem_u32(qbuf) + warp * 4096;
        float* dst = whole ? a.part_o : reinterpret_cast<float*>(piece);
        const int my_row = !live ? -1 : whole ? (int)out_row : rr;
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
          float o[32];
          tmem_ld32(to + 32 * c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = inv == 0.f ? 0.f : o[j] * w0;
          if (second) {
            float x[32];
            tmem_ld32(to + 128 + 32 * c, x);
            tmem_wait_ld32(x);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = fmaf(x[j], w1, o[j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sts128(stage + lane * 128 + ((j ^ (lane & 7)) << 4),
                   make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]), __float_as_uint(o[4 * j + 2]),
                              __float_as_uint(o[4 * j + 3])));
          __syncwarp();
          const int e = 32 * c + 4 * (lane & 7);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = 4 * j + (lane >> 3), row = __shfl_sync(0xffffffffu, my_row, k);
            const uint4 v = lds128(stage + k * 128 + (((lane & 7) ^ (k & 7)) << 4));
            if (row >= 0 && e < a.D) *reinterpret_cast<uint4*>(dst + (size_t)row * a.D + e) = v;
          }
          __syncwarp();
        }
      }
      tc_before();
      named_barrier<256>(1);  // both streams' outputs and `other` have been read
    }
  } else if (warp < 16) {
    registers_down<kOtherRegs>();
    // ------------------------------------------------ keys (warps 8-11) and values (12-15): 16 codes a thread and load,
    // as fp16 tiles
    const int t = tid & 127, ch = t & 3, tk = t >> 2 & (S::kTokens - 1), half = S::kHalves == 2 ? t >> 6 : 0;
    const int e = half * 64 + ch * 16;
    const bool in = e < a.D, values = warp >= 12;
    const uint8_t* cache = static_cast<const uint8_t*>(values ? a.v_cache : a.k_cache) + e;
    uint64_t* full = values ? v_full : k_full;
    uint4 raw[S::kLoads];
    // the next step's loads, what is not there as zeros; they are on the way while this step's MMAs run
    int i = 0;
    bool more = next_segment(sg, step);
    auto fetch = [&]() {
      const int slot = (sg.g + i) % kSlots, seen = in ? ctxs[sg.item.r] - (sg.tok0 + i * TOK) : 0;
      if (!wait_warp(found + slot, (sg.g + i) / kSlots & 1)) return false;
#pragma unroll
      for (int k = 0; k < S::kLoads; ++k) {
        const int tok = k * S::kTokens + tk;
        const long long base = unit_at[slot][tok / kUnit];
        raw[k] = load_if(cache + base + (tok % kUnit) * a.D, base >= 0 && tok < seen);
      }
      if (++i == sg.n) i = 0, more = next_segment(sg, step);
      return true;
    };
    bool ok = !more || fetch();
    uint8_t* tiles = (values ? vbuf : kbuf) + half * S::kBlock;
#pragma unroll 1
    for (int g = 0; ok && g < share.c1 - share.c0; ++g) {
      const int b = g & 1;
      // the products of two steps ago have read the tile
      ok = g < 2 || (values ? wait_warp(spent + (g - 2) % kSlots, (g - 2) / kSlots & 1)
                            : wait_warp(k_empty + b, ((g >> 1) - 1) & 1));
      if (!ok) break;
      // rows of 64 elements, 16-byte chunks swizzled; eight lanes are the four chunk pairs of two tokens: no conflicts
      const uint32_t dst = smem_u32(tiles) + b * S::kTile;
#pragma unroll
      for (int k = 0; k < S::kLoads; ++k) {
        const int tok = k * S::kTokens + tk;
        uint4 f[2];
        codes_to_f16<FMT>(raw[k].x, f[0].x, f[0].y);
        codes_to_f16<FMT>(raw[k].y, f[0].z, f[0].w);
        codes_to_f16<FMT>(raw[k].z, f[1].x, f[1].y);
        codes_to_f16<FMT>(raw[k].w, f[1].z, f[1].w);
#pragma unroll
        for (int j = 0; j < 2; ++j) sts128(dst + tok * 128 + (((2 * ch + j) ^ (tok & 7)) << 4), f[j]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + b);
      if (more) ok = fetch();
    }
  } else if (warp == 16) {
    registers_down<kOtherRegs>();
    // ------------------------------------------------ a lane per unit of 16 tokens: its block and the block's scales
    const float2* scales = reinterpret_cast<const float2*>(a.scales);
    bool ok = true;
    while (ok && next_segment(sg, step)) {
      const int ctx = ctxs[sg.item.r];
      auto look = [&](int i) {
        const int tok = sg.tok0 + i * TOK + lane * kUnit;
        int blk = -1;
        if (i < sg.n && lane < kUnits && tok < ctx) {
          blk = a.table[(size_t)sg.item.r * a.max_blocks + tok / a.bs];
          if (blk < 0 || blk >= a.num_blocks) {
            report_error(a.err, kErrKvBlock);
            blk = -1;
          }
        }
        return blk;
      };
      auto scales_of = [&](int blk) {
        return blk >= 0 ? scales[(size_t)blk * a.Hkv + sg.item.h] : make_float2(0.f, 1.f);
      };
      int blk = look(0);
#pragma unroll 1
      for (int i = 0; i < sg.n; ++i) {
        const int g = sg.g + i, slot = g % kSlots;
        ok = g < kSlots || wait_warp(spent + slot, (g / kSlots - 1) & 1);
        if (!ok) break;
        if (lane < kUnits) {
          const int row = (sg.tok0 + i * TOK + lane * kUnit) % a.bs;
          unit_at[slot][lane] = blk < 0 ? -1 : (((long long)blk * a.Hkv + sg.item.h) * a.bs + row) * a.D;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(found + slot);
        const float2 sc = scales_of(blk);
        const int next = look(i + 1);
        if (lane < kUnits) {
          // a value scale below 2^-64 counts as 2^-64; what comes off the sum is what went on
          const float lv = __log2f(sc.y < kMinScale ? kMinScale : sc.y);
          unit_scales[slot][lane] = make_float4(sc.x, lv, ex2(-lv), blk < 0 ? 0.f : sc.y == 0.f ? 2.f : 1.f);
        }
        const bool usual = __all_sync(0xffffffffu, lane >= kUnits || (blk >= 0 && sc.y != 0.f));
        if (lane == 0) plain[slot] = usual;
        __syncwarp();
        if (lane == 0) mbar_arrive(scaled + slot);
        blk = next;
      }
    }
  } else if (warp > 17) {
    registers_down<kOtherRegs>();
  } else {
    registers_down<kOtherRegs>();
    // ------------------------------------------------ MMAs
    // What decides the loops and forms the operands is taken from lane 0, so that it stays in uniform registers.
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t one = lane == 0, is = tc_idesc(128, TOK, false, false), io = tc_idesc(128, DP, false, true);
    const uint32_t tb = uniform(tbase);
    const uint64_t qd = tc_desc(uniform(smem_u32(qbuf)), 16, 1024), kd = tc_desc(uniform(smem_u32(kbuf)), 16, 1024),
                   vd = tc_desc(uniform(smem_u32(vbuf)), S::kBlock, 1024);
    uint32_t passes0 = 0, passes1 = 0;  // of p_ready
    bool ok = true;
    while (ok && __all_sync(0xffffffffu, next_segment(sg, step))) {
      const int n = uniform(sg.n), gi = uniform(sg.g), two = uniform(sg.rows > kRowsTile);
      const int events = two ? 2 * n : n;  // event x: stream x & 1, of step x / 2 or x
      // (a wait costs this warp some 200 cycles of the 1450 that an event's products take: each is made once, where it is
      // not in the way)
      auto keys_there = [&](int x) {
        const int g = gi + (two ? x >> 1 : x), b = g & 1;
        return (two && (x & 1)) || wait_warp(k_full + b, (g >> 1) & 1);
      };
      auto issue_s = [&](int x) {
        const int t = x & 1, g = gi + (two ? x >> 1 : x), b = g & 1;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t at = ((k >> 2) * S::kBlock + (k & 3) * 32) >> 4;
          mma_ss(tb + S::kColS + 128 * t, qd + at + (t * S::kTile >> 4), kd + at + (b * S::kTile >> 4), is, k > 0, one);
        }
        if (one) {
          tc_commit(s_full + t);
          if (!two || t == 1) tc_commit(k_empty + b);
        }
        __syncwarp();
      };
      ok = wait_warp(&q_full, uniform(sg.index) & 1);
      ok = ok && keys_there(0) && (events < 2 || two || keys_there(1));
      if (!ok) break;
      tc_after();
      issue_s(0);
      if (events > 1) issue_s(1);
#pragma unroll 1
      for (int x = 0; ok && x < events; ++x) {
        const int t = x & 1, g = gi + (two ? x >> 1 : x), b = g & 1;
        ok = ((two && t) || wait_warp(v_full + b, (g >> 1) & 1)) && (x + 2 >= events || keys_there(x + 2)) &&
             wait_warp(p_ready + t, (t ? passes1 : passes0) & 1);
        if (!ok) break;
        (t ? passes1 : passes0) += 1;
        tc_after();
#pragma unroll
        for (int k = 0; k < TOK / 16; ++k)
          mma_ts(tb + S::kColO + 128 * t, tb + S::kColS + 128 * t + 8 * k, vd + ((b * S::kTile + k * 2048) >> 4), io,
                 k > 0 ? 1u : x > 1, one);
        if (one && (!two || t == 1)) tc_commit(spent + g % kSlots);
        __syncwarp();
        if (x + 2 < events) issue_s(x + 2);
      }
      if (one) tc_commit(&o_done);
      __syncwarp();
    }
  }
  if (tid == 0) pdl_wait();
  // After a wait that gave up: the products in flight end before the memory is given back (a bounded wait).
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 17) {
    if (abort_flag) {
      if (lane == 0) {
        tc_commit(&o_done);
        for (int ph = 0; ph < 2; ++ph) mbar_wait_n(&o_done, ph, nullptr, 0, 1u << 14);
      }
      __syncwarp();
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u));
  }
}

template <int FMT, int DP>
cudaError_t launch(const AttnArgs& a, uint8_t* pieces, int2* source, int ctas, cudaStream_t stream, bool pdl) {
  auto k = attn_kv8_prefix_kernel<FMT, DP>;
  const cudaError_t e = allow_max_smem(k);
  if (e != cudaSuccess) return e;
  return launch_kernel(k, dim3(ctas), dim3(kThreads), PrefixShape<DP>::kSmem + 16 * ((size_t)a.R + 1), stream, pdl, a,
                       pieces, source);
}

}  // namespace

cudaError_t launch_attn_kv8_prefix(const AttnArgs& a, int format, uint8_t* pieces, int2* source, int ctas,
                                   cudaStream_t stream, bool pdl) {
  if (format == QG_KV_I8)
    return a.D <= 64 ? launch<QG_KV_I8, 64>(a, pieces, source, ctas, stream, pdl)
                     : launch<QG_KV_I8, 128>(a, pieces, source, ctas, stream, pdl);
  return a.D <= 64 ? launch<QG_KV_E4M3, 64>(a, pieces, source, ctas, stream, pdl)
                   : launch<QG_KV_E4M3, 128>(a, pieces, source, ctas, stream, pdl);
}

}  // namespace qg
