// Attention of a step's query tokens over the paged 8-bit key/value cache, with
// warp-level matrix instructions: up to 16 query rows (query tokens times the
// query heads of a group) per pass over the cache.
//
//   t = (q . k) (ks scale log2 e) + log2(vs)    k, v: codes; ks, vs: the block's scales
//   p = 2^(t - m),  acc += p v,  l += p / vs,   out = acc / l
//
// The value scale enters through the exponent, so codes are multiplied as they
// are: int8 and e4m3 are exact in fp16, and so is q after an exact power of two
// per row; p is rounded to fp16 (2^-11 relative), everything else is fp32. The
// running maximum m moves only when a score passes it by 2^8: p stays below
// 2^8, far inside fp16, and a step without such a score scales nothing.
//
// The cache is read once, so HBM bounds it: the GPU's steps (of 256 tokens of a
// key/value head) are dealt to one CTA per SM in equal shares, wherever a
// context begins or ends; each of a CTA's 8 warps takes 32 tokens of a step
// through a TMA ring of its own (no barrier between warps until an item ends).
// Keys come out of the swizzled ring as A fragments of S^T = K q^T, values
// through ldmatrix's byte transposition as A fragments of O^T = V^T P^T: nothing
// is converted twice and nothing goes back to shared memory. Pieces of a context
// cut by shares are added up by the CTA that brings the last one.
// Measured (32 query heads, 8 key/value heads of 128, int8): 131071 tokens 50.5 us,
// 268 MB at 5.3 TB/s; the streaming itself runs at 6.7 TB/s, and 10 us go to the
// launch, the first copies and the joining of pieces. 32 requests of 1..8192
// tokens (e4m3): 52.8 us, 270 MB. One token over 37 tokens: 6.4 us, all latency.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_kv8.cuh"
#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

// An item costs about as much as 2 steps to begin and end; one of up to 3 steps is not cut: joining its pieces takes
// longer than its steps on one CTA. With (2, 3), (3, 6) and (1, 3): 32 ragged requests of four drafts 65.1, 68.3 and
// 73.7 us, of one token 52.8, 54.2 and 56.6; one of 1024 tokens 8.9, 10.3 and 8.8; 16 of 1..1024 tokens 11.3, 11.1, 15.5.
constexpr int kItemCost = 2;
constexpr int kWholeSteps = 3;

// D: elements of a head, filled up with zeros to 64, 128 or 256 as the copies land (a.D is what the arrays have)
template <int D, int NT, int FMT>
struct AttnShape {
  static constexpr int kWarps = 8;
  static constexpr int kRows = 8 * NT;
  static_assert(kRows <= kMmaRows, "the workspace's pieces");
  static constexpr int kUps = NT <= 2 && D <= 128 ? 2 : 1;  // units of a warp's step
  static constexpr int kSubs = D > 128 ? D / 128 : 1;  // 128-byte column blocks of a token
  static constexpr int kRowBytes = D > 128 ? 128 : D;
  static constexpr int kHalves = D / 64;               // 64-byte steps of q . k
  static constexpr int kMt = D / 16;                   // 16-row tiles of the output's transpose
  static constexpr int kUnitBytes = kUnit * D;         // a unit's keys (or values)
  static constexpr int kStage = 2 * kUps * kUnitBytes; // a step's keys, then its values
  static constexpr int kStepTokens = kUnit * kUps * kWarps;
  static constexpr int kPass = NT == 1 ? 4 : 8;        // output tiles that the warps' parts are added up of at a time
  static constexpr int kBuf = kWarps * kPass * 32 * 16;
  static constexpr bool kQRegs = NT * kHalves <= 4;    // the query fragments stay in registers
  static constexpr int kQ = kQRegs ? 0 : kHalves * 4 * NT * 32 * 8;
  static constexpr int kRaw = 2 * kRows * D * 2;
};

// Order of a unit's tokens. ldmatrix with 8-bit transposition gives lane (g, c)
// of a 16 x 16 tile the elements d = g (and g + 8) of the tokens of its rows
// 4 c .. 4 c + 3: the value product's A operand with MMA columns 2 c, 2 c + 1, 2 c + 8,
// 2 c + 9 = rows 4 c .. 4 c + 3, so MMA row i of the scores' product is row
// 4 (i % 8 / 2) + i % 2 + 2 (i / 8). Row -> token: rows that one shared-memory
// phase touches together must differ in the address bits that the swizzle does
// not already spread: D >= 128 (128-byte rows, chunk ^= row & 7) pairs rows that
// differ by 4, D = 64 (64-byte rows, chunk ^= row / 2 & 3) odd with even.
template <int D>
__device__ __forceinline__ int unit_token(int row) {
  const int b0 = row & 1, b1 = row >> 1 & 1, b2 = row >> 2 & 1;
  return D == 64 ? row : (row & 8) | (b0 ^ b2) << 2 | b1 << 1 | b2;
}

// byte offset of 16-byte chunk `ch` of token row `row` in a swizzled [16][kRowBytes] tile
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int row, int ch) {
  return D == 64 ? row * 64 + ((ch ^ (row >> 1 & 3)) << 4) : row * 128 + ((ch ^ (row & 7)) << 4);
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}
// two 16 x 16 byte tiles, transposed: see unit_token
__device__ __forceinline__ void ldmatrix_t8(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int D, int NT, int FMT>
__global__ void __launch_bounds__(32 * AttnShape<D, NT, FMT>::kWarps, 1)
    attn_kv8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs a,
                    int stages, uint32_t ring_offset, int wide) {
  using S = AttnShape<D, NT, FMT>;
  constexpr int NW = S::kWarps, ROWS = S::kRows, UPS = S::kUps, TOK = S::kStepTokens;
  using Cut = AttnCut<TOK, kItemCost, kWholeSteps>;
  constexpr int SB = 32 / UPS;  // steps whose units the lanes look after
  extern __shared__ __align__(1024) uint8_t smem[];
  // layout: ring | combine buffer | q fragments | rows | warp maxima and sums | meta | barriers | batch
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem;
  uint8_t* p = smem + (size_t)ring_offset;
  float4* buf = reinterpret_cast<float4*>(p);
  p += S::kBuf;
  uint2* qfrag = reinterpret_cast<uint2*>(p);  // [half * 4 + word][nt][lane]
  p += S::kQ;
  uint8_t* qraw = p;  // [2][ROWS][D] bf16: this segment's queries and the next one's
  p += S::kRaw;
  // rows of the item, a copy per warp: tokens below .x are seen, and draft tokens by .y's bits; .z: output row or -1
  int4* row_info = reinterpret_cast<int4*>(p) + warp * ROWS;
  p += 16 * NW * ROWS;
  float2* wstat = reinterpret_cast<float2*>(p);  // [NW][ROWS] maxima and sums
  p += 8 * NW * ROWS;
  float4* meta = reinterpret_cast<float4*>(p);  // [NW][stages][UPS] key scale, log2 and inverse of the value scale, kind
  p += 16 * NW * stages * UPS;
  uint64_t* bars = reinterpret_cast<uint64_t*>(p);  // [NW][stages]
  p += 8 * NW * stages;
  int* first = reinterpret_cast<int*>(p);  // [R + 1]
  int* cost = first + a.R + 1;             // [R + 1]
  int* cus = cost + a.R + 1;               // [R + 1]
  int* ctxs = cus + a.R + 1;               // [R]
  __shared__ int2 scan_part[NW];
  __shared__ unsigned arrived;
  __shared__ float row_factor[ROWS];

  if (lane == 0)
#pragma unroll 1
    for (int s = 0; s < stages; ++s) mbar_init(bars + warp * stages + s, 1);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();

  const int G = a.Hq / a.Hkv;
  const AttnBatch batch = attn_scan<ROWS, Cut, 32 * NW>(a, first, cost, cus, ctxs, scan_part);
  const AttnShare mine_of = attn_share<Cut>(batch, a.err);
  const int c0 = mine_of.c0, c1 = mine_of.c1, n = c1 - c0;
  if (n == 0) return;

  // the queries of the item that `at` lies in, to buffer `b` (asynchronous)
  auto fetch_q = [&](const AttnPlace& at, int b) {
    const int q_first = cus[at.r], rows = (cus[at.r + 1] - q_first) * G;
#pragma unroll 1
    for (int i = threadIdx.x; i < ROWS * (D / 8); i += 32 * NW) {
      const int rr = i / (D / 8), rho = at.rt * ROWS + rr;
      const bool live = rho < rows && 8 * (i % (D / 8)) < a.D;
      const uint16_t* src = a.q;
      if (live) src += (q_first + rho / G) * a.q_stride + (at.h * G + rho % G) * a.D + 8 * (i % (D / 8));
      cp_async16(smem_u32(qraw + (size_t)b * ROWS * D * 2 + 16 * i), src, live);
    }
  };
  AttnPlace ahead = attn_locate<ROWS, Cut>(batch, c0);  // of the next segment
  fetch_q(ahead, 0);

  // ---- producer side of the warp's ring: a lane looks after one unit of SB steps ----
  uint64_t* bar = bars + warp * stages;
  float4* my_meta = meta + warp * stages * UPS;
  uint8_t* my_ring = ring + (size_t)warp * stages * S::kStage;
  int page = -1, row = 0;
  float4 scale = make_float4(0.f, 0.f, 0.f, 0.f);
  int n_blk = -1, n_head = 0, n_row = 0;  // of the following batch of steps
  float2 n_scale = make_float2(0.f, 0.f);
  auto look_table = [&](int b) {
    n_blk = -1;
    const int step = c0 + SB * b + lane / UPS;
    if (step < c1) {
      const AttnPlace at = attn_locate<ROWS, Cut>(batch, step);
      const int tok = ((at.s * NW + warp) * UPS + lane % UPS) * kUnit;
      if (tok < ctxs[at.r]) {
        n_blk = a.table[(size_t)at.r * a.max_blocks + tok / a.bs];
        n_head = at.h;
        n_row = tok % a.bs;
        if (n_blk < 0 || n_blk >= a.num_blocks) {
          report_error(a.err, kErrKvBlock);
          n_blk = -1;
        }
      }
    }
  };
  auto look_scale = [&]() {
    if (n_blk >= 0)
      n_scale = reinterpret_cast<const float2*>(a.scales)[(size_t)n_blk * a.Hkv + n_head];
  };
  auto next_batch = [&]() {
    page = n_blk >= 0 ? n_blk * a.Hkv + n_head : -1;
    row = n_row;
    // a value scale below 2^-64 counts as 2^-64: what it adds to an output is below 2^-55; of a block of zero
    // scale only the probabilities count
    const float v = n_scale.y < kMinScale ? kMinScale : n_scale.y;
    scale = make_float4(n_scale.x, __log2f(v), __frcp_rn(v), page < 0 ? 0.f : n_scale.y == 0.f ? 2.f : 1.f);
  };
  // the first batch's pages are known before its scales: the copies of the first steps do not wait for them
  auto first_batch = [&]() {
    page = n_blk >= 0 ? n_blk * a.Hkv + n_head : -1;
    row = n_row;
  };
  auto issue = [&](int i, int slot) {
    const int k = i & (SB - 1);
    if (k == 0 && i > 0) {
      next_batch();
      look_table(i / SB + 1);
    }
    if (k == SB / 2) look_scale();
    if (i >= stages && lane / UPS == k) my_meta[slot * UPS + lane % UPS] = scale;  // the warp reads it after a barrier of its own
    int pages[UPS], rows[UPS], units = 0;
#pragma unroll
    for (int u = 0; u < UPS; ++u) {
      pages[u] = __shfl_sync(0xffffffffu, page, k * UPS + u);
      rows[u] = __shfl_sync(0xffffffffu, row, k * UPS + u);
      units += pages[u] >= 0 ? 1 : 0;
    }
    if (lane == 0) {
      const uint32_t dst = smem_u32(my_ring + (size_t)slot * S::kStage);
      uint64_t* b = bar + slot;
      if (units == 0) {
        mbar_arrive(b);
      } else if (UPS == 2 && wide) {
        // both units lie in one block (or the second one past the context, in the block all the same)
        mbar_arrive_expect_tx(b, S::kStage);
        tma_load_3d(dst, &kmap, 0, rows[0], pages[0], b);
        tma_load_3d(dst + UPS * S::kUnitBytes, &vmap, 0, rows[0], pages[0], b);
      } else {
        mbar_arrive_expect_tx(b, 2 * units * S::kUnitBytes);
#pragma unroll
        for (int u = 0; u < UPS; ++u) {
          if (pages[u] >= 0) {
#pragma unroll
            for (int sub = 0; sub < S::kSubs; ++sub) {
              const uint32_t at = dst + u * S::kUnitBytes + sub * kUnit * S::kRowBytes;
              tma_load_3d(at, &kmap, sub * 128, rows[u], pages[u], b);
              tma_load_3d(at + UPS * S::kUnitBytes, &vmap, sub * 128, rows[u], pages[u], b);
            }
          }
        }
      }
    }
  };
  look_table(0);
  look_scale();
  first_batch();

  // ---- consumer ----
  float acc[NT][S::kMt][4];
  float m[NT][2], l[NT][2], rf[NT][2];
  constexpr bool kQRegs = S::kQRegs;
  uint2 qr[kQRegs ? S::kHalves * 4 : 1][kQRegs ? NT : 1];
  AttnPlace item = {};
  int seg_end = c0, item_first = c0;
  int ctx = 0, nq = 0, q0 = 0, base = 0;
  bool ok = true;

  int qb = 0;
  auto begin_segment = [&](int step) {
    item = ahead;
    item_first = step - item.s;
    seg_end = min(c1, item_first + item.steps);
    ctx = ctxs[item.r];
    q0 = cus[item.r];
    nq = cus[item.r + 1] - q0;
    base = ctx - nq;
    const bool tree = a.tree && nq <= 32;
#pragma unroll 1
    for (int rr = lane; rr < ROWS; rr += 32) {
      const int rho = item.rt * ROWS + rr;
      int4 info = make_int4(0, 0, -1, 0);
      if (rho < nq * G) {
        const int i = rho / G;
        info.x = tree ? base : base + i + 1;
        if (tree) info.y = (int)(a.tree[q0 + i] & (0xFFFFFFFFu >> (32 - nq)));
        info.z = (q0 + i) * a.Hq + item.h * G + rho - i * G;
      }
      row_info[rr] = info;
    }
    cp_async_wait_all();
    __syncthreads();
    // q as the B operand: 2^-sigma q in fp16, exact, sigma per row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (kQRegs || nt % NW == warp) {
        const uint8_t* src = qraw + ((size_t)qb * ROWS + nt * 8 + g) * D * 2 + 32 * c;
        uint4 raw[S::kHalves][2];
        float amax = 0.f;
#pragma unroll
        for (int hf = 0; hf < S::kHalves; ++hf) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            raw[hf][k] = *reinterpret_cast<const uint4*>(src + 128 * hf + 16 * k);
            const uint32_t w[4] = {raw[hf][k].x, raw[hf][k].y, raw[hf][k].z, raw[hf][k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float x = __uint_as_float(w[j] << 16), y = __uint_as_float(w[j] & 0xFFFF0000u);
              amax = fmaxf(amax, fmaxf(fabsf(x), fabsf(y)));
            }
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int sigma = fp16_prescale_exp(amax);
        const float down = pow2f(-sigma), up = a.scale_log2 * pow2f(sigma);
        if (kQRegs) {
          rf[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);
          rf[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
        } else if (c == 0) {
          row_factor[nt * 8 + g] = up;
        }
#pragma unroll
        for (int hf = 0; hf < S::kHalves; ++hf) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint4 u = raw[hf][w >> 1];
            const uint32_t x = w & 1 ? u.z : u.x, y = w & 1 ? u.w : u.y;
            const uint2 f = make_uint2(f16x2(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down),
                                       f16x2(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xFFFF0000u) * down));
            if (kQRegs)
              qr[hf * 4 + w][nt] = f;
            else
              qfrag[((hf * 4 + w) * NT + nt) * 32 + lane] = f;
          }
        }
      }
    }
    if (!kQRegs) __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (!kQRegs) rf[nt][j] = row_factor[nt * 8 + 2 * c + j];
        m[nt][j] = kNoMax;
        l[nt][j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][mt][j] = 0.f;
    }
    // the other buffer was last read before the barrier above
    qb ^= 1;
    if (seg_end < c1) {
      ahead = attn_locate<ROWS, Cut>(batch, seg_end);
      fetch_q(ahead, qb);
    }
  };

  // lane's places in a swizzled tile: keys (token t0; t0 + 2 is 2 rows on), values (ldmatrix rows)
  const int t0 = unit_token<D>(4 * (g >> 1) + (g & 1)), t1 = t0 + 2;
  const uint32_t k_at0 = tile_offset<D>(t0, c), k_at1 = tile_offset<D>(t1, c);
  const uint32_t v_at = tile_offset<D>(unit_token<D>(lane & 15), lane >> 4);

  // the step's units, landed at `stage`; the first one's first token is `tok`
  auto compute = [&](uint32_t stage, const float4 (&mu)[UPS], int tok) {
    float s[UPS][NT][4];
#pragma unroll
    for (int u = 0; u < UPS; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[u][nt][j] = 0.f;
      // S^T = K q^T: lane (g, c) holds tokens t0, t1 and 16-byte chunk c of each 64 bytes
#pragma unroll
      for (int hf = 0; hf < S::kHalves; ++hf) {
        const uint32_t tile = stage + u * S::kUnitBytes + (hf >> 1) * kUnit * S::kRowBytes, x = 64 * (hf & 1);
        const uint4 k0 = lds128((tile + k_at0) ^ x), k1 = lds128((tile + k_at1) ^ x);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t f[4];
          codes_to_f16<FMT>(w0[w], f[0], f[2]);
          codes_to_f16<FMT>(w1[w], f[1], f[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = kQRegs ? qr[hf * 4 + w][nt] : qfrag[((hf * 4 + w) * NT + nt) * 32 + lane];
            mma16816(s[u][nt], f, b.x, b.y);
          }
        }
      }
    }
    // t = log2 of (probability times value scale); lane: tokens t0, t1 of rows 2 c, 2 c + 1
    bool grow = false, edge[UPS];
    uint32_t keep[UPS];
#pragma unroll
    for (int u = 0; u < UPS; ++u) {
      const int at0 = tok + u * kUnit;
      // some row may not see some token, or the unit is absent or has no values
      edge[u] = at0 + kUnit > base || mu[u].w != 1.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[u][nt][j] = fmaf(s[u][nt][j], mu[u].x * rf[nt][j & 1], mu[u].y);
      if (edge[u]) {
        keep[u] = 0u;  // bytes of the lane's value words that count (slots past the context may hold no numbers)
        if (mu[u].w == 1.f) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (at0 + unit_token<D>(4 * c + b) < ctx) keep[u] |= 0xFFu << (8 * b);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int at = at0 + (j < 2 ? t0 : t1);
            const unsigned d = (unsigned)(at - base);
            const int2 lim = *reinterpret_cast<const int2*>(row_info + nt * 8 + 2 * c + (j & 1));
            const bool seen = mu[u].w != 0.f && (at < lim.x || (d < 32u && ((unsigned)lim.y >> d & 1u)));
            if (!seen) s[u][nt][j] = -INFINITY;
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        // (the difference, which is exact where it is small: m + kSlack may round up to a score whose p passes fp16)
        grow |= fmaxf(s[u][nt][0], s[u][nt][2]) - m[nt][0] > kSlack ||
                fmaxf(s[u][nt][1], s[u][nt][3]) - m[nt][1] > kSlack;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
          if (UPS == 2) x = fmaxf(x, fmaxf(s[UPS - 1][nt][j], s[UPS - 1][nt][j + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[nt][j], x), f = ex2(m[nt][j] - mn);
          m[nt][j] = mn;
          l[nt][j] *= f;
#pragma unroll
          for (int mt = 0; mt < S::kMt; ++mt) acc[nt][mt][j] *= f, acc[nt][mt][j + 2] *= f;
        }
      }
    }
    uint32_t pb[UPS][NT][2];
#pragma unroll
    for (int u = 0; u < UPS; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = ex2(s[u][nt][j] - m[nt][j & 1]);
        l[nt][0] = fmaf(e[0] + e[2], mu[u].z, l[nt][0]);
        l[nt][1] = fmaf(e[1] + e[3], mu[u].z, l[nt][1]);
        // (token, row) -> (row, token): the B operand of the value product
        pb[u][nt][0] = transpose8x8(f16x2(e[0], e[1]));
        pb[u][nt][1] = transpose8x8(f16x2(e[2], e[3]));
      }
    }
    // O^T += V^T p^T, two 16-element tiles of the head at a time
#pragma unroll
    for (int u = 0; u < UPS; ++u) {
#pragma unroll
      for (int k = 0; k < S::kMt / 2; ++k) {
        const uint32_t tile = stage + (UPS + u) * S::kUnitBytes + k / 4 * kUnit * S::kRowBytes;
        uint32_t v[4];
        ldmatrix_t8((tile + v_at) ^ (32 * (k % 4)), v);
        if (edge[u]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] &= keep[u];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t f[4];
          codes_to_f16<FMT>(v[2 * i], f[0], f[2]);
          codes_to_f16<FMT>(v[2 * i + 1], f[1], f[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(acc[nt][2 * k + i], f, pb[u][nt][0], pb[u][nt][1]);
        }
      }
    }
  };

  // result of tile q = nt * kMt + mt: lane (g, c) holds elements d = 16 mt + g and d + 8 of rows 2 c, 2 c + 1 as
  // {d r0, d r1, d+8 r0, d+8 r1}; l0, l1 the rows' sums, 0 where no token is seen (the result is 0 then). Lanes of
  // even and odd g trade a row each, so that a lane writes pairs.
  auto write_out = [&](int q, const float4 o, float l0, float l1) {
    const int nt = q / S::kMt, mt = q - nt * S::kMt, odd = g & 1;
    const float i0 = l0 == 0.f ? 0.f : __frcp_rn(l0), i1 = l1 == 0.f ? 0.f : __frcp_rn(l1);
    const float x0 = o.x * i0, x1 = o.y * i1, y0 = o.z * i0, y1 = o.w * i1;
    const float x = __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 4), y = __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 4);
    const int to = row_info[nt * 8 + 2 * c + odd].z;
    if (to >= 0 && 16 * mt < a.D) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + (size_t)to * a.D + 16 * mt + (g & 6));
      dst[0] = odd ? f32_to_bf16x2(x, x1) : f32_to_bf16x2(x0, x);
      dst[4] = odd ? f32_to_bf16x2(y, y1) : f32_to_bf16x2(y0, y);
    }
  };

  constexpr int kTiles = NT * S::kMt;
  auto end_segment = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
        if (g == 0) wstat[warp * ROWS + nt * 8 + 2 * c + j] = make_float2(m[nt][j], l[nt][j]);
      }
    }
    const bool whole = item_first >= c0 && item_first + item.steps <= c1;
    uint8_t* ws = static_cast<uint8_t*>(a.ws) + kAttnCounterBytes;
    // a CTA has a piece of at most two items: one begun before its share, one that goes on after it
    uint8_t* mine = ws + (size_t)(2 * blockIdx.x + (item_first < c0 ? 0 : 1)) * attn_piece_bytes(ROWS, D);
    float4* stat = reinterpret_cast<float4*>(mine + (size_t)ROWS * D * 4);
    // In the CTA's last segment the ring is free: all tiles at once there, else S::kPass at a time.
    const bool last = seg_end == c1 && stages * S::kStage * NW >= NW * kTiles * 512;
    float4* sum_buf = last ? reinterpret_cast<float4*>(ring) : buf;
    const int per_pass = last ? kTiles : S::kPass;
    __syncthreads();
    // to the item's maximum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mm[2] = {kNoMax, kNoMax};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(wstat + w * ROWS + nt * 8 + 2 * c);
        mm[0] = fmaxf(mm[0], x.x), mm[1] = fmaxf(mm[1], x.z);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float f = ex2(m[nt][j] - mm[j]);
#pragma unroll
        for (int mt = 0; mt < S::kMt; ++mt) acc[nt][mt][j] *= f, acc[nt][mt][j + 2] *= f;
      }
    }
    // all warps' parts into shared memory, then a tile per warp is added up
#pragma unroll 1
    for (int t0 = 0; t0 < kTiles; t0 += per_pass) {
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        if (last || q / S::kPass * S::kPass == t0)
          sum_buf[(warp * per_pass + q - t0) * 32 + lane] =
              make_float4(acc[q / S::kMt][q % S::kMt][0], acc[q / S::kMt][q % S::kMt][1], acc[q / S::kMt][q % S::kMt][2],
                          acc[q / S::kMt][q % S::kMt][3]);
      }
      __syncthreads();
#pragma unroll 1
      for (int q = t0 + warp; q < t0 + per_pass; q += NW) {
        const int nt = q / S::kMt, mt = q - nt * S::kMt;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float mm[2] = {kNoMax, kNoMax}, ll[2] = {0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 x = sum_buf[(w * per_pass + q - t0) * 32 + lane];
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
          const float4 y = *reinterpret_cast<const float4*>(wstat + w * ROWS + nt * 8 + 2 * c);
          mm[0] = fmaxf(mm[0], y.x), mm[1] = fmaxf(mm[1], y.z);
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(wstat + w * ROWS + nt * 8 + 2 * c);
          ll[0] = fmaf(y.y, ex2(y.x - mm[0]), ll[0]), ll[1] = fmaf(y.w, ex2(y.z - mm[1]), ll[1]);
        }
        if (whole) {
          write_out(q, o, ll[0], ll[1]);
        } else {
          reinterpret_cast<float4*>(mine)[q * 32 + lane] = o;
          if (mt == 0 && g == 0) stat[nt * 4 + c] = make_float4(mm[0], ll[0], mm[1], ll[1]);
        }
      }
      if (t0 + per_pass < kTiles) __syncthreads();
    }
    if (whole) return;
    // the CTA that brings an item's last piece adds the pieces up, in the order of the CTAs
    const int f = attn_cta_of<Cut>(batch, mine_of, item_first),
              e = attn_cta_of<Cut>(batch, mine_of, item_first + item.steps - 1), pieces = e - f + 1;
    unsigned* count = static_cast<unsigned*>(a.ws) + f;
    __syncthreads();  // (thread 0's release and acquire stand for the whole CTA's accesses on either side)
    if (threadIdx.x == 0) {
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(arrived) : "l"(count) : "memory");
      if (arrived == (unsigned)(e - f)) *count = 0u;  // the next call finds it as this one did
    }
    __syncthreads();
    if (arrived != (unsigned)(e - f)) return;
    // Factors of the pieces, a row per warp; then a tile per warp (or several warps, each a part of the pieces), whose
    // first loads are on their way meanwhile.
    float* factor = reinterpret_cast<float*>(buf);  // [pieces][ROWS]
    auto piece = [&](int i) {
      return ws + (size_t)(2 * (f + i) + (i == 0 ? 1 : 0)) * attn_piece_bytes(ROWS, D);
    };
    // (as many as the registers allow without the main loop feeling it: 8192 tokens 12.1 us with 8, 11.6 with 20)
    constexpr int kParts = kTiles < NW ? NW / kTiles : 1, kEarly = NT == 1 && D <= 128 ? 20 : 8;
    const int part = kParts > 1 ? warp / kTiles : 0;
    float4 early[kEarly];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) {
      const int i = part + k * kParts;
      early[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < pieces) early[k] = __ldcg(reinterpret_cast<const float4*>(piece(i)) + warp % kTiles * 32 + lane);
    }
#pragma unroll 1
    for (int rr = warp; rr < ROWS; rr += NW) {
      float2 st[kMaxCtas / 32];
      float mm = kNoMax, ll = 0.f;
#pragma unroll
      for (int k = 0; k < kMaxCtas / 32; ++k) {
        const int i = lane + 32 * k;
        st[k] = i < pieces ? __ldcg(reinterpret_cast<const float2*>(piece(i) + (size_t)ROWS * D * 4) + rr)
                           : make_float2(kNoMax, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kMaxCtas / 32; ++k) mm = fmaxf(mm, st[k].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
#pragma unroll
      for (int k = 0; k < kMaxCtas / 32; ++k) {
        const float x = ex2(st[k].x - mm);
        if (lane + 32 * k < pieces) factor[(lane + 32 * k) * ROWS + rr] = x;
        ll = fmaf(st[k].y, x, ll);
      }
      ll = warp_sum(ll);
      if (lane == 0) wstat[rr].y = ll;
    }
    __syncthreads();
#pragma unroll 1
    for (int q = warp % kTiles, from = part + kEarly * kParts; q < kTiles; q += NW, from = part) {
      const int rr = q / S::kMt * 8 + 2 * c;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (from != part) {
#pragma unroll
        for (int k = 0; k < kEarly; ++k) {
          const int i = part + k * kParts;
          if (i < pieces) {
            const float2 fa = *reinterpret_cast<const float2*>(factor + i * ROWS + rr);
            o.x = fmaf(early[k].x, fa.x, o.x), o.y = fmaf(early[k].y, fa.y, o.y);
            o.z = fmaf(early[k].z, fa.x, o.z), o.w = fmaf(early[k].w, fa.y, o.w);
          }
        }
      }
#pragma unroll 8
      for (int i = from; i < pieces; i += kParts) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(piece(i)) + q * 32 + lane);
        const float2 fa = *reinterpret_cast<const float2*>(factor + i * ROWS + rr);
        o.x = fmaf(x.x, fa.x, o.x), o.y = fmaf(x.y, fa.y, o.y);
        o.z = fmaf(x.z, fa.x, o.z), o.w = fmaf(x.w, fa.y, o.w);
      }
      if (kParts > 1) {
        __syncthreads();
        buf[warp * 32 + lane] = o;
        __syncthreads();
        if (part) break;
#pragma unroll 1
        for (int k = 1; k < kParts; ++k) {
          const float4 x = buf[(warp + k * kTiles) * 32 + lane];
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
      }
      write_out(q, o, wstat[rr].y, wstat[rr + 1].y);
    }
  };

  // Iteration i issues step i + stages and consumes step i; the first ones only issue. (Every larger part of the
  // loop stands in the code once: its size is what a cold start waits for.)
  int slot = 0, tok = 0;
  uint32_t phase = 1;
#pragma unroll 1
  for (int i = -stages;; ++i) {
    if (i >= 0) {
      if (i == n || c0 + i == seg_end) {
        if (i > 0) end_segment();
        if (i == n) break;
        if (i == 0) {
          // the first batch's scales have arrived; its first steps' ones go where issue() puts the others'
          next_batch();
          if (lane / UPS < stages) my_meta[lane] = scale;
          look_table(1);
        }
        begin_segment(c0 + i);
        tok = (item.s * NW + warp) * UPS * kUnit;
      }
      if (ok && !__all_sync(0xffffffffu, mbar_try_wait(bar + slot, phase)))
        ok = __all_sync(0xffffffffu, mbar_wait(bar + slot, phase, a.err, kErrAttnWait));
      if (ok) {
        float4 mu[UPS];
        bool any = false;
#pragma unroll
        for (int u = 0; u < UPS; ++u) mu[u] = my_meta[slot * UPS + u], any |= mu[u].w != 0.f;
        if (any) compute(smem_u32(my_ring + (size_t)slot * S::kStage), mu, tok);
        __syncwarp();
      }
      tok += TOK;
    }
    if (ok && i + stages < n) issue(i + stages, slot);
    if (++slot == stages) slot = 0, phase ^= 1u;
  }
  if (!ok)  // the copies still in flight land before the shared memory is given up (bounded waits)
#pragma unroll 1
    for (int s = 0; s < stages; ++s) mbar_wait_n(bar + s, phase, nullptr, 0, 1u << 16);
}

struct AttnLaunch {
  int stages;
  uint32_t ring;
  size_t smem;
};
template <int D, int NT, int FMT>
AttnLaunch attn_smem(int R) {
  using S = AttnShape<D, NT, FMT>;
  const size_t fixed = S::kBuf + S::kQ + S::kRaw + 24 * S::kWarps * S::kRows + 16 * (size_t)(R + 1);
  const size_t budget = (size_t)device_max_smem_optin() - 2048 - fixed;
  const size_t per = (size_t)S::kWarps * (S::kStage + 16 * S::kUps + 8);
  AttnLaunch l;
  // Two steps ahead (128 KB an SM) are enough to stream at HBM's rate; more only queue up there, and CTAs end further
  // apart (131071 tokens 51.7 us with three, 50.6 with two; e4m3 51.3 and 49.8; heads of 256, 65536 tokens 54.7 and 53.8;
  // 32 ragged requests 57.8 and 57.0; only with e4m3 in blocks of 16 the other way, 52.3 and 52.8).
  l.stages = (int)std::min<size_t>(2, budget / per);
  l.ring = (uint32_t)((size_t)l.stages * S::kWarps * S::kStage);
  l.smem = fixed + per * l.stages;
  return l;
}

// steps of all items, at most (8 rows, 128 tokens); the kernel counts them in 32 bits
long long attn_most_steps(const AttnArgs& a) {
  const long long tiles = ((long long)a.T * (a.Hq / a.Hkv)) / 8 + 2LL * a.R;
  return tiles * a.Hkv * (((long long)a.max_blocks * a.bs + 127) / 128 + 1 + 8);
}

template <int D, int NT, int FMT>
cudaError_t launch_mma(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  using S = AttnShape<D, NT, FMT>;
  CUtensorMap km, vm;
  const int wide = S::kUps == 2 && a.bs % 32 == 0;  // a step's two units in one box
  const auto sw = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  for (int i = 0; i < 2; ++i)
    if (!tmap_3d(i ? &vm : &km, CU_TENSOR_MAP_DATA_TYPE_UINT8, i ? a.v_cache : a.k_cache, a.D, a.bs,
                 (uint64_t)a.num_blocks * a.Hkv, a.D, (uint64_t)a.bs * a.D, S::kRowBytes, wide ? 2 * kUnit : kUnit, 1, sw))
      return cudaErrorInvalidValue;
  auto k = attn_kv8_kernel<D, NT, FMT>;
  cudaError_t e = allow_max_smem(k);
  if (e != cudaSuccess) return e;
  const AttnLaunch l = attn_smem<D, NT, FMT>(a.R);
  return launch_kernel(k, dim3(std::min(device_sm_count(), kMaxCtas)), dim3(32 * S::kWarps), l.smem, stream, pdl, km, vm, a, l.stages,
                       l.ring, wide);
}

// the width a head of D elements is filled up to
int attn_width(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// rows of an average request's item
int attn_rows(const AttnArgs& a) { return (int)(((long long)a.T + a.R - 1) / a.R) * (a.Hq / a.Hkv); }
// The tcgen05 kernel for many rows of up to 128 elements. This file's kernel passes over the cache once per 16 rows, at
// 5 ns per 128 tokens of a head (3 ns with heads of 64); that one takes 7 ns per 128 tokens and 64 rows, and about 3 us
// more to begin, end and join. Measured, here and there: one request, 64 rows, 300 tokens 9.5 and 14.0 us, 2048 tokens
// 14.5 and 15.0, 8192 tokens 23.9 and 18.1, 32784 tokens 57.2 and 30.8; 32 rows, 8192 tokens 16.7 and 16.9, 32768 tokens
// 34.3 and 28.2; heads of 64, 64 rows, 65536 tokens 41.4 and 30.7; six requests of 40 rows over 5000 tokens 11.8 and
// 15.8. The lengths are known to the GPU alone, so their bound decides: short contexts of a table made for long ones
// take the longer time.
bool attn_tc_ok(const AttnArgs& a) {
  const int width = attn_width(a.D);
  if (width > kTcHead) return false;
  const long long rows = attn_rows(a), steps = (long long)a.R * a.Hkv * (((long long)a.max_blocks * a.bs + 127) / 128);
  return steps * ((width == 64 ? 3 : 5) * ((rows + 15) / 16) - 7 * ((rows + 63) / 64)) >= 3000;
}

// 8-row tiles per item: the least that hold an average request's query rows
template <int FMT>
cudaError_t launch_by_shape(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  const bool one = attn_rows(a) <= 8;
  switch (attn_width(a.D)) {
    case 64: return one ? launch_mma<64, 1, FMT>(a, stream, pdl) : launch_mma<64, 2, FMT>(a, stream, pdl);
    case 128: return one ? launch_mma<128, 1, FMT>(a, stream, pdl) : launch_mma<128, 2, FMT>(a, stream, pdl);
    default: return one ? launch_mma<256, 1, FMT>(a, stream, pdl) : launch_mma<256, 2, FMT>(a, stream, pdl);
  }
}

}  // namespace

size_t attn_kv8_workspace_size(int, int, int D) {
  // which kernel runs depends on the call: the larger pieces of those that may
  size_t piece = attn_piece_bytes(kMmaRows, attn_width(D));
  if (attn_width(D) <= kTcHead) piece = std::max(piece, attn_piece_bytes(kTcRows, kTcHead));
  return kAttnCounterBytes + 2 * (size_t)std::min(device_sm_count(), kMaxCtas) * piece;
}

bool attn_kv8_ok(const AttnArgs& a) { return attn_most_steps(a) < (1LL << 31); }

cudaError_t launch_attn_kv8(const AttnArgs& a, int format, cudaStream_t stream, bool pdl) {
  if (attn_tc_ok(a)) return launch_attn_kv8_tc(a, format, stream, pdl);
  return format == QG_KV_I8 ? launch_by_shape<QG_KV_I8>(a, stream, pdl) : launch_by_shape<QG_KV_E4M3>(a, stream, pdl);
}

}  // namespace qg
