// Attention over the paged 8-bit cache for many query rows per key/value head of
// up to 128 elements (more than 16 rows: drafts of a speculative tree, or a prompt's
// piece, times the heads of a group), on the 5th-generation tensor cores.
//
// The warp-level kernel of attn_kv8.cu reads the cache once for every 16 rows.
// Here a step of 128 tokens is read and converted once for up to 64:
//   S^T [128 tokens][N rows] = K q^T    A = the keys as fp16 in TMEM (a thread
//       converts a token's row and stores it to its own lane), B = the queries;
//   P^T = 2^(S^T ... - m)               a thread per token, half of the rows: what is a
//       maximum over the tokens becomes a test against the row's m, so no
//       exchange between threads unless some score outgrows m by 2^8;
//   O^T [128][N rows] += V^T P^T          A = the values as fp16 in shared memory,
//       token-major as converted (MN-major operand), B = P^T as written.
// The value scale of a token's block enters through the exponent and comes off
// the sum again, as in attn_kv8.cu. Sums, maxima and accumulators are fp32, K, V
// and q are exact in fp16, p is rounded to fp16.
//
// Sixteen warps per CTA, one CTA per SM: 0-3 convert keys and half of the values,
// 4-7 and 8-11 softmax of half of the rows each, 12 and 13 the values' other half,
// 14 issues the copies, 15 the MMAs (16 warps are what leaves a thread 128
// registers). Steps run through two
// buffers of every kind; S of step i + 1 is issued before O of step i. The batch
// is cut into shares as in attn_kv8.cu; a second kernel joins a context's pieces.
//
// Measured: 64 rows of 8 heads over 32784 int8 tokens 30.8 us (67 MB at 2.2 TB/s, 8.6
// GFLOP), 65568 tokens 48 us. A step takes 1.26 us against 0.6 us of copies (a 152nd of
// HBM) and 0.3 us of MMAs: it is bound by the chain from one S to its P in the softmax
// warps and by what the MMA warp waits for and issues, all at about 2300 cycles; no single
// part taken out makes it more than 8 % faster. 6 us go to the first step, 5 to the last
// results and their joining.
#include <cuda_runtime.h>

#include <algorithm>

#include "attn_kv8.cuh"
#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kTcTok = 128;     // tokens of a step
constexpr int kTcThreads = 512;
// an item costs about 7 us to begin and end, a step 1.25 us; joining is a kernel of its own, so only the shortest items
// are kept whole
using TcCut = AttnCut<kTcTok, 5, 2>;
constexpr int kTcMaxCtas = 152;  // CTAs: the join kernel's factors and the table of split items are laid out for it

constexpr int D = kTcHead;  // elements of a head; fewer (a.D) are filled up with zeros as the copies land
struct TcShape {
  static constexpr int kTile = kTcTok * D;                // a step's keys (or values) as stored
  static constexpr int kStage = 2 * kTile;
  static constexpr int kV = kTcTok * D * 2;               // a step's values as fp16: [2][128 tokens][64]
  static constexpr int kP = kTcTok * kTcRows * 2;         // [128 tokens][64 rows] fp16
  static constexpr int kQ = kTcRows * D * 2;              // [2][64 rows][64] fp16
  static constexpr int kColK = 0, kColS = 2 * (D / 2), kColO = kColS + 2 * kTcRows;  // TMEM columns
};
constexpr uint32_t kTcCols = 512;

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle, version 1. K-major: rows of
// 64 fp16, `sbo` bytes between groups of 8 rows (lbo unused). MN-major: rows are
// K, 64 contiguous fp16 of M or N each; sbo between groups of 8 K rows, lbo
// between blocks of 64 M (N).
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// instruction descriptor: fp16 operands, fp32 accumulator
__device__ __forceinline__ constexpr uint32_t tc_idesc(int M, int N, bool a_mn, bool b_mn) {
  return 1u << 4 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
// Issued where `one` is set (one lane), by code that the whole warp runs: descriptors are then uniform registers.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                       uint32_t one) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// sixteen columns of the thread's lane, to be touched after tmem_wait_ld
__device__ __forceinline__ void tmem_ld16(uint32_t t, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(t));
}
__device__ __forceinline__ void tmem_wait_ld(float* v) {  // orders later uses of v[0..15] after the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}

template <int COUNT>
__device__ __forceinline__ void named_barrier(int id) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(COUNT) : "memory");
}
template <int COUNT>
__device__ __forceinline__ bool named_barrier_or(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(p ? 1u : 0u), "r"(id), "n"(COUNT)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float x) { return pair2(__float_as_uint(x), __float_as_uint(x)); }
// the larger of R values over the 32 lanes, as transposed_warp_sum: lane L gets that of value transposed_row<R>(L)
template <int R>
__device__ __forceinline__ float transposed_warp_max(float (&v)[R], int lane) {
  int cnt = R;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (cnt > 1) {
      const int half = cnt / 2;
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < R / 2; ++i) {
        if (i < half) {
          const float keep = upper ? v[i + half] : v[i], send = upper ? v[i] : v[i + half];
          v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
      }
      cnt = half;
    } else {
      v[0] = fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
    }
  }
  return v[0];
}

constexpr unsigned kRowSpan = 16u << 23;  // rows' queries that differ by 2^16, on the bits of fp32, do not share a scale
constexpr int kTcMaxStages = 3;
// Slots of the scales of a step: when step h's are written the values of step h - 3 have been converted, and before them
// the P of step h - 5 was read: the softmax is at step h - 4 or later.
constexpr int kTcSlots = 8;

// one entry per CTA, behind the counters of attn_kv8.cu's pieces
__device__ __forceinline__ int4* tc_splits(void* ws) {
  return reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + kMaxCtas * 4);
}
static_assert(kMaxCtas * 4 + kTcMaxCtas * 16 <= kAttnCounterBytes, "");
static_assert(kTcMaxCtas <= kMaxCtas, "the workspace has pieces for kMaxCtas");

// the rest of a wait that did not succeed at once; gives up when another role has
__device__ __noinline__ bool tc_wait_on(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* err) {
#pragma unroll 1
  for (uint32_t i = 0; i < kMaxPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  report_error(err, kErrAttnWait);
  *abort_flag = 1u;
  return false;
}

// Elements 64 part .. 64 part + 63 of token t's values, from the tile at src to fp16 rows of 64 at dst; zeros where
// there is no token (slots past the context may hold codes that are not numbers).
template <int FMT>
__device__ __forceinline__ void tc_values(uint32_t src, uint32_t dst, int part, int t, bool none) {
  dst += part * kTcTok * 128 + t * 128;
  src += t * 128;
#pragma unroll
  for (int ch = 0; ch < 4; ++ch) {
    const uint4 w = lds128(src + (((4 * part + ch) ^ (t & 7)) << 4));
    uint4 f[2];
    codes_to_f16<FMT>(w.x, f[0].x, f[0].y);
    codes_to_f16<FMT>(w.y, f[0].z, f[0].w);
    codes_to_f16<FMT>(w.z, f[1].x, f[1].y);
    codes_to_f16<FMT>(w.w, f[1].z, f[1].w);
#pragma unroll
    for (int k = 0; k < 2; ++k) sts128(dst + (((2 * ch + k) ^ (t & 7)) << 4), f[k]);
  }
  if (none)
#pragma unroll 1
    for (int ch = 0; ch < 8; ++ch) sts128(dst + (ch << 4), make_uint4(0u, 0u, 0u, 0u));
}

template <int FMT>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_kv8_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, AttnArgs a,
                       int box, int stages) {
  using S = TcShape;
  constexpr int ROWS = kTcRows, TOK = kTcTok;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, role = warp >> 2, quad = warp & 3;
  uint8_t* ring = smem;
  uint8_t* vbuf = ring + stages * S::kStage;
  uint8_t* pbuf = vbuf + 2 * S::kV;
  uint8_t* qbuf = pbuf + 2 * S::kP;
  int* first = reinterpret_cast<int*>(qbuf + S::kQ);
  int* cost = first + a.R + 1;
  int* cus = cost + a.R + 1;
  int* ctxs = cus + a.R + 1;
  __shared__ __align__(16) float neg_m[ROWS], fall[ROWS], fade[ROWS], sums[ROWS];
  __shared__ __align__(16) float wsum[4][ROWS];
  __shared__ int4 row_info[ROWS];  // tokens below .x are seen, and draft tokens by .y's bits; .z: output row or -1
  __shared__ uint64_t full[kTcMaxStages], empty[kTcMaxStages], s_full[2], o_done[2], q_full;
  // s_ready: the step's keys are in TMEM and the scores of two steps ago have been read; o_ready: its P and values are there
  __shared__ uint64_t s_ready[2], o_ready[2];
  __shared__ uint64_t scaled[kTcSlots];  // the step's scales have been written
  __shared__ float4 unit_scales[kTcSlots][TOK / kUnit];
  __shared__ int2 scan_part[kTcThreads / 32];
  __shared__ uint32_t tmem_base;
  __shared__ __align__(16) float row_scale[ROWS];  // factors of scores, where the rows' queries differ in scale
  __shared__ unsigned amax_bits, amin_bits;  // the rows' largest finite |q|: the largest and the smallest above 0
  __shared__ unsigned unset_any[2];
  __shared__ volatile uint32_t abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kTcMaxStages; ++i) mbar_init(full + i, 1), mbar_init(empty + i, 6);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_ready + i, 4 + 8);
      mbar_init(s_full + i, 1);
      mbar_init(o_ready + i, 8 + 6);
      mbar_init(o_done + i, 1);
    }
    mbar_init(&q_full, 8);
    for (int i = 0; i < kTcSlots; ++i) mbar_init(scaled + i, 1);
    abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                 "r"(kTcCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_before();
  const AttnBatch batch = attn_scan<ROWS, TcCut, kTcThreads>(a, first, cost, cus, ctxs, scan_part);  // has barriers
  tc_after();
  const AttnShare share = attn_share<TcCut>(batch, a.err);
  const uint32_t tbase = tmem_base;
  const uint32_t tlane = tbase + ((uint32_t)(quad * 32) << 16);  // the lanes that this warp may touch

  // by a whole warp, which goes on together
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) ||
           __all_sync(0xffffffffu, tc_wait_on(bar, parity, &abort_flag, a.err));
  };

  // A segment: the steps of one item in this CTA's share. Every role walks the segments by itself; buffers and
  // barriers run on from one to the next (step g of the CTA: buffer g & 1), so the keys and values of a segment are
  // converted while the last one's results are written.
  struct Segment {
    AttnPlace item;
    int n, g, ctx, q0, nq, base, rows, nch, tok0, item_first, index;  // nch: 16 nch columns are in use
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
    s.item = attn_locate<ROWS, TcCut>(batch, step);
    s.item_first = step - s.item.s;
    s.n = min(share.c1, s.item_first + s.item.steps) - step;
    s.ctx = ctxs[s.item.r];
    s.q0 = cus[s.item.r];
    s.nq = cus[s.item.r + 1] - s.q0;
    s.base = s.ctx - s.nq;
    s.rows = min(ROWS, s.nq * batch.G - s.item.rt * ROWS);
    s.nch = (s.rows + 15) / 16;
    s.tok0 = s.item.s * TOK;
    return true;
  };
  int4 split = make_int4(0, 0, 0, 0);  // pieces | rows << 16, first query token, head, row tile
  int st = 0;  // ring stage of a role's next step, and the parity of its passes through the ring
  uint32_t pass = 0;
  int step = share.c0;
  Segment sg = first_segment();
  if (role == 0) {
    // ------------------------------------------------ keys: a token's row per thread, fp16 into TMEM; half of its values
    const int t = quad * 32 + lane;
    bool ok = true;
    while (ok && next_segment(sg, step)) {
#pragma unroll 1
      for (int i = 0; i < sg.n; ++i) {
        const int g = sg.g + i, b = g & 1;
        ok = wait_warp(full + st, pass) && (g < 2 || wait_warp(s_full + b, ((g >> 1) - 1) & 1));
        if (!ok) break;  // S of two steps ago has read the buffer
        tc_after();
        const uint32_t src = smem_u32(ring + (size_t)st * S::kStage);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t f[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int ch = 4 * h + j;
            const uint32_t at = t * 128 + ((ch ^ (t & 7)) << 4);
            const uint4 w = lds128(src + at);
            codes_to_f16<FMT>(w.x, f[8 * j], f[8 * j + 1]);
            codes_to_f16<FMT>(w.y, f[8 * j + 2], f[8 * j + 3]);
            codes_to_f16<FMT>(w.z, f[8 * j + 4], f[8 * j + 5]);
            codes_to_f16<FMT>(w.w, f[8 * j + 6], f[8 * j + 7]);
          }
          tmem_st32(tlane + S::kColK + b * (D / 2) + 32 * h, f);
        }
        tmem_wait_st();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_ready + b);
        // half of the token's values
        ok = g < 2 || wait_warp(o_done + b, ((g >> 1) - 1) & 1);
        if (!ok) break;
        tc_values<FMT>(src + S::kTile, smem_u32(vbuf + b * S::kV), 0, t, sg.tok0 + i * TOK + t >= sg.ctx);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st), mbar_arrive(o_ready + b);
        if (++st == stages) st = 0, pass ^= 1u;
      }
    }
  } else if (warp == 12 || warp == 13) {
    // ------------------------------------------------ values: the other half of two tokens' per thread, fp16 into shared memory
    bool ok = true;
    while (ok && next_segment(sg, step)) {
#pragma unroll 1
      for (int i = 0; i < sg.n; ++i) {
        const int g = sg.g + i, b = g & 1;
        ok = wait_warp(full + st, pass) && (g < 2 || wait_warp(o_done + b, ((g >> 1) - 1) & 1));
        if (!ok) break;
        const uint32_t src = smem_u32(ring + (size_t)st * S::kStage + S::kTile);
#pragma unroll 1
        for (int t = (warp - 12) * 32 + lane; t < TOK; t += 64)
          tc_values<FMT>(src, smem_u32(vbuf + b * S::kV), 1, t, sg.tok0 + i * TOK + t >= sg.ctx);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st), mbar_arrive(o_ready + b);
        if (++st == stages) st = 0, pass ^= 1u;
      }
    }
  } else if (warp == 14) {
    // ------------------------------------------------ copies: `box` tokens of one block at a time
    // A lane looks after a unit of 16 tokens: its block, and what the softmax needs of the block's scales (one warp
    // works it out; two more warps of every quarter would otherwise look up each token: 1 of their 9 instructions).
    const int boxes = TOK / box, per_box = box / kUnit;
    const float2* scales = reinterpret_cast<const float2*>(a.scales);
    bool ok = true;
    while (ok && next_segment(sg, step)) {
      auto look = [&](int i) {
        const int tok = sg.tok0 + i * TOK + lane * kUnit;
        int blk = -1;
        if (i < sg.n && lane < TOK / kUnit && tok < sg.ctx) {
          blk = a.table[(size_t)sg.item.r * a.max_blocks + tok / a.bs];
          if (blk < 0) blk = a.num_blocks;  // bad
        }
        return blk;
      };
      auto scales_of = [&](int blk) {
        return blk >= 0 && blk < a.num_blocks ? scales[(size_t)blk * a.Hkv + sg.item.h] : make_float2(0.f, -1.f);
      };
      int blk = look(0), next = look(1);
      float2 sc = scales_of(blk);
#pragma unroll 1
      for (int i = 0; i < sg.n; ++i) {
        const int g = sg.g + i, mine = __shfl_sync(0xffffffffu, blk, lane * per_box & 31);
        ok = g < stages || wait_warp(empty + st, pass ^ 1u);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(full + st, S::kStage);
        __syncwarp();
        if (lane < boxes) {
          if (mine >= a.num_blocks) report_error(a.err, kErrKvBlock);
          // what is not there is read past the last page: zeros
          const int page = mine >= 0 && mine < a.num_blocks ? mine * a.Hkv + sg.item.h : a.num_blocks * a.Hkv;
          const int row = (sg.tok0 + i * TOK + lane * box) % a.bs;
          const uint32_t dst = smem_u32(ring + (size_t)st * S::kStage) + lane * box * D;
          tma_load_3d(dst, &kmap, 0, row, page, full + st);
          tma_load_3d(dst + S::kTile, &vmap, 0, row, page, full + st);
        }
        if (lane < TOK / kUnit) {
          // key scale, log2 of the value scale and 2^-that (not its inverse: what comes off is what went on), kind
          const float lv = __log2f(sc.y < kMinScale ? kMinScale : sc.y);
          unit_scales[g % kTcSlots][lane] =
              make_float4(sc.x, lv, ex2(-lv), sc.y == 0.f ? 2.f : sc.y > 0.f || sc.y != sc.y ? 1.f : 0.f);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(scaled + g % kTcSlots);
        blk = next;
        next = look(i + 2);
        sc = scales_of(blk);
        if (++st == stages) st = 0, pass ^= 1u;
      }
    }
  } else if (warp == 15) {
    // ------------------------------------------------ MMAs
    // What decides the loops and forms the operands is taken from lane 0, so that all of it stays in uniform registers:
    // otherwise this warp's instructions bound the step (16 MMAs and their waits 2700 cycles).
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t io = tc_idesc(D, ROWS, true, true), one = lane == 0;
    const uint32_t tb = uniform(tbase), qs = uniform(smem_u32(qbuf)), vs = uniform(smem_u32(vbuf)), ps = uniform(smem_u32(pbuf));
    const uint64_t qd = tc_desc(qs, 16, 1024), vd = tc_desc(vs, TOK * 128, 1024), pd = tc_desc(ps, TOK * 128, 1024);
    bool ok = true;
    while (ok && __all_sync(0xffffffffu, next_segment(sg, step))) {
      const int n = uniform(sg.n), gi = uniform(sg.g);
      const uint32_t is = tc_idesc(128, 16 * uniform(sg.nch), false, false);
      ok = wait_warp(&q_full, uniform(sg.index) & 1);
#pragma unroll 1
      for (int i = 0; i <= n && ok; ++i) {
        if (i < n) {
          const uint32_t g = gi + i, b = g & 1;
          ok = wait_warp(s_ready + b, (g >> 1) & 1);
          if (!ok) break;
          tc_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ts(tb + S::kColS + b * ROWS, tb + S::kColK + b * (D / 2) + 8 * k,
                   qd + (((k >> 2) * ROWS * 128 + (k & 3) * 32) >> 4), is, k > 0, one);
          if (one) tc_commit(s_full + b);
          __syncwarp();
        }
        if (i > 0) {
          const uint32_t g = gi + i - 1, b = g & 1;
          ok = wait_warp(o_ready + b, (g >> 1) & 1);
          if (!ok) break;
          tc_after();
#pragma unroll
          for (int k = 0; k < TOK / 16; ++k)
            mma_ss(tb + S::kColO, vd + ((b * S::kV + k * 2048) >> 4), pd + ((b * S::kP + k * 2048) >> 4), io,
                   k > 0 ? 1u : i > 1, one);
          if (one) tc_commit(o_done + b);
          __syncwarp();
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax: a token per thread, half of the rows
    constexpr int HR = ROWS / 2;
    if (lane == 0) mbar_arrive(s_ready), mbar_arrive(s_ready + 1);  // both buffers of S are free
    const int t = quad * 32 + lane, half = role == 1 ? 0 : 1, bar = 1 + half;
    while (next_segment(sg, step)) {
      const AttnPlace item = sg.item;
      const int n = sg.n, gi = sg.g, base = sg.base, tok0 = sg.tok0, nch = sg.nch, rows = sg.rows;
      // The item's queries: 2^-sigma q in fp16, K-major, swizzled; four threads a row. One sigma serves the item's rows
      // (its largest finite |q| just below 2^15) down to rows 2^-16 of that, whose values keep 2^-24 of the row's
      // largest; a smaller row gets a sigma of its own and its scores a factor. What is not finite stays so, in its own
      // row's products. (The last segment's products have been waited for.)
      const int u = half * 128 + t;
      float up;
      auto rows_differ = [&]() {  // some row has a sigma of its own
        return amin_bits < amax_bits && amax_bits - amin_bits > kRowSpan;
      };
      {
        constexpr int kPer = 256 / ROWS, kTimes = D / 8 / kPer;  // threads of a row, 8 elements at a time
        const int rr = u / kPer, c0 = u % kPer, rho = item.rt * ROWS + rr, qi = rho / batch.G;
        const int head = item.h * batch.G + rho - qi * batch.G;
        uint4 raw[kTimes];
        const uint16_t* src = a.q + (size_t)(sg.q0 + qi) * a.q_stride + head * a.D;
#pragma unroll
        for (int k = 0; k < kTimes; ++k) {
          const int ch = c0 + k * kPer;
          raw[k] = make_uint4(0u, 0u, 0u, 0u);
          if (rr < rows && 8 * ch < a.D) raw[k] = *reinterpret_cast<const uint4*>(src + 8 * ch);
        }
        if (u == 0) amax_bits = 0u, amin_bits = 0xFFFFFFFFu;
        if (c0 == 0) {
          int4 info = make_int4(0x7FFFFFFF, 0, -1, 0);
          if (rr < rows) {
            const bool tree = a.tree && sg.nq <= 32;
            info.x = tree ? base : base + qi + 1;
            if (tree) info.y = (int)(a.tree[sg.q0 + qi] & (0xFFFFFFFFu >> (32 - sg.nq)));
            info.z = (sg.q0 + qi) * a.Hq + head;
          }
          row_info[rr] = info;
          neg_m[rr] = 0.f;
        }
        named_barrier<256>(3);
        unsigned row_max = 0u;  // largest finite |q| as the bits of an fp32
#pragma unroll
        for (int k = 0; k < kTimes; ++k) {
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned lo = w[j] << 16 & 0x7FFF0000u, hi = w[j] & 0x7FFF0000u;
            row_max = max(row_max, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
          }
        }
#pragma unroll
        for (int o = 1; o < kPer; o <<= 1) row_max = max(row_max, __shfl_xor_sync(0xffffffffu, row_max, o));
        const unsigned most = __reduce_max_sync(0xffffffffu, row_max),
                       least = __reduce_min_sync(0xffffffffu, row_max ? row_max : 0xFFFFFFFFu);
        if (lane == 0) atomicMax(&amax_bits, most), atomicMin(&amin_bits, least);
        named_barrier<256>(3);
        int sigma = fp16_prescale_exp(__uint_as_float(amax_bits));
        up = a.scale_log2 * pow2f(sigma);
        const bool differ = rows_differ();
        if (differ) {
          int own = sigma;
          if (row_max && amax_bits - row_max > kRowSpan)
            own = max(fp16_prescale_exp(__uint_as_float(row_max)), sigma - 126);
          if (c0 == 0) row_scale[rr] = pow2f(own - sigma);
          sigma = own;
        }
        const float down = pow2f(-sigma);
#pragma unroll
        for (int k = 0; k < kTimes; ++k) {
          const int ch = c0 + k * kPer;
          const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
          uint32_t f[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            f[j] = f16x2(__uint_as_float(w[j] << 16) * down, __uint_as_float(w[j] & 0xFFFF0000u) * down);
          sts128(smem_u32(qbuf) + (ch >> 3) * ROWS * 128 + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                 make_uint4(f[0], f[1], f[2], f[3]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
        if (differ) named_barrier<256>(3);
      }
      // this half's columns: hch chunks of 16 from column hc on
      const int hc = half ? 16 * ((nch + 1) / 2) : 0, hch = half ? nch / 2 : (nch + 1) / 2;
      const uint32_t t_s = tlane + S::kColS + hc, t_o = tlane + S::kColO + hc;
      float* nm_of = neg_m + hc;
      uint64_t l[HR / 2];  // sums of columns 2 j, 2 j + 1
#pragma unroll
      for (int j = 0; j < HR / 2; ++j) l[j] = 0ull;
      bool unset = true;  // some row has seen no token yet
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int g = gi + i, b = g & 1, tok = tok0 + i * TOK + t;
        wait_warp(scaled + g % kTcSlots, g / kTcSlots & 1);
        const float4 sc = unit_scales[g % kTcSlots][t / kUnit];
        const uint64_t ks2 = both(sc.x * up), lv2 = both(sc.y), inv2 = both(sc.z);
        const bool there = sc.w != 0.f, zero = sc.w == 2.f, edge = __any_sync(0xffffffffu, !there || tok >= base);
        // (After a wait that gave up every later one returns at once: the warps stay in step at their barriers.)
        uint64_t c[HR / 2];  // log2 of the value scale, less the row's m
#pragma unroll
        for (int j = 0; j < HR; j += 4) {
          const ulonglong2 nm = *reinterpret_cast<const ulonglong2*>(nm_of + j);
          c[j / 2] = fadd2(lv2, nm.x), c[j / 2 + 1] = fadd2(lv2, nm.y);
        }
        // (all of them here: loaded one after the other where they are used they take 0.3 us of a step)
#pragma unroll
        for (int j = 0; j < HR / 2; ++j) asm volatile("" : "+l"(c[j]));
        wait_warp(s_full + b, (g >> 1) & 1);
        tc_after();
        float y[HR];
#pragma unroll
        for (int ch = 0; ch < HR / 16; ++ch)
          if (ch < hch) tmem_ld16(t_s + b * ROWS + 16 * ch, y + 16 * ch);
#pragma unroll
        for (int ch = 0; ch < HR / 16; ++ch)
          if (ch < hch) tmem_wait_ld(y + 16 * ch);
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_ready + b);
        bool grow = unset;
#pragma unroll
        for (int j = 0; j < HR; j += 2)
          if (j / 16 < hch)
            unpair2(ffma2(pair2(__float_as_uint(y[j]), __float_as_uint(y[j + 1])), ks2, c[j / 2]), y[j], y[j + 1]);
        if (edge) {
          // which rows see the token (a rolled loop: this code is met once or twice and has to be fetched)
          const unsigned d = (unsigned)(tok - base);
          uint32_t seen = 0u;
#pragma unroll 2
          for (int j = 0; j < 16 * hch; ++j) {
            const int2 lim = *reinterpret_cast<const int2*>(row_info + hc + j);
            seen |= (tok < lim.x || (d < 32u && ((unsigned)lim.y >> d & 1u)) ? 1u : 0u) << j;
          }
          if (!there) seen = 0u;
#pragma unroll
          for (int j = 0; j < HR; ++j)
            if (j / 16 < hch) y[j] = seen >> j & 1u ? y[j] : -INFINITY;
        }
        float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < HR; j += 8) {
          if (j / 16 < hch) {
#pragma unroll
            for (int k = 0; k < 4; ++k) most[k] = fmaxf(fmaxf(most[k], y[j + k]), y[j + k + 4]);
          }
        }
        grow |= fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) > kSlack;
        // (P of two steps ago has been read: its product was issued before this step's S, whose end has been waited for)
        if (named_barrier_or<128>(bar, grow)) {
          // rows with a sigma of their own: the factor for what the scores put on top of c (here, where such items come
          // in every step, and not where scores are read: the loop has no register to spare, 64 rows over 65568 tokens
          // took 57 us instead of 48)
          if (rows_differ()) {
#pragma unroll
            for (int j = 0; j < HR; ++j) {
              if (j / 16 < hch) {
                const float cj = sc.y + nm_of[j];
                y[j] = fmaf(row_scale[hc + j], y[j] - cj, cj);
              }
            }
          }
          // rows whose m has to rise (or to be set): the largest y over the step's tokens
          {
            float top[HR];
#pragma unroll
            for (int j = 0; j < HR; ++j) top[j] = j / 16 < hch ? y[j] : -INFINITY;
            const float x = transposed_warp_max<HR>(top, lane);
            const int j = transposed_row<HR>(lane);
            if (j < 16 * hch) wsum[quad][hc + j] = x;
          }
          if (t == 0) unset_any[half] = 0u;
          named_barrier<128>(bar);
          if (t < 16 * hch) {
            const int j = hc + t;
            const float top = fmaxf(fmaxf(wsum[0][j], wsum[1][j]), fmaxf(wsum[2][j], wsum[3][j]));
            const bool is_set = row_info[j].w != 0;
            // a first maximum may be below 0 (nothing has been summed yet), a later one only raises m
            const float rise = top == -INFINITY ? 0.f : is_set ? fmaxf(top, 0.f) : top;
            if (!is_set && top != -INFINITY) row_info[j].w = 1;
            if (!is_set && top == -INFINITY) unset_any[half] = 1u;
            fall[j] = -rise;
            fade[j] = ex2(fminf(-rise, 0.f));
            neg_m[j] -= rise;
          }
          named_barrier<128>(bar);
          unset = unset_any[half] != 0u || rows_differ();
          if (i > 0) wait_warp(o_done + ((g - 1) & 1), ((g - 1) >> 1) & 1);
          tc_after();
#pragma unroll
          for (int j = 0; j < HR; j += 4) {
            if (j / 16 < hch) {
              const float4 r = *reinterpret_cast<const float4*>(fall + hc + j);
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(fade + hc + j);
              y[j] += r.x, y[j + 1] += r.y, y[j + 2] += r.z, y[j + 3] += r.w;
              l[j / 2] = ffma2(l[j / 2], f.x, 0ull);
              l[j / 2 + 1] = ffma2(l[j / 2 + 1], f.y, 0ull);
            }
          }
          if (i > 0) {
#pragma unroll 1
            for (int ch = 0; ch < hch; ++ch) {
              float o[16];
              tmem_ld16(t_o + 16 * ch, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= fade[hc + 16 * ch + j];
              tmem_st16(t_o + 16 * ch, o);
            }
          }
          if (i > 0) tmem_wait_st();
          tc_before();
        }
        // p, its sum without the value scale, and as fp16 in shared memory (of a block of zero scale nothing)
        const uint32_t dst = smem_u32(pbuf + b * S::kP) + t * 128;
        const bool some_zero = __any_sync(0xffffffffu, zero);
#pragma unroll
        for (int c8 = 0; c8 < HR / 8; ++c8) {
          if (c8 / 2 < hch) {
            uint32_t f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = 8 * c8 + 2 * k;
              const float e0 = ex2(y[j]), e1 = ex2(y[j + 1]);
              l[j / 2] = ffma2(pair2(__float_as_uint(e0), __float_as_uint(e1)), inv2, l[j / 2]);
              f[k] = f16x2(e0, e1);
            }
            if (some_zero) {
#pragma unroll
              for (int k = 0; k < 4; ++k) f[k] = zero ? 0u : f[k];
            }
            sts128(dst + (((c8 + hc / 8) ^ (t & 7)) << 4), make_uint4(f[0], f[1], f[2], f[3]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_ready + b);
      }
      // the rows' sums over the tokens: per warp, then over the warps
      {
        float part[HR];
#pragma unroll
        for (int j = 0; j < HR / 2; ++j) unpair2(l[j], part[2 * j], part[2 * j + 1]);
        const float x = transposed_warp_sum<HR>(part, lane);
        const int j = transposed_row<HR>(lane);
        if (j < 16 * hch) wsum[quad][hc + j] = x;
      }
      const int item_first = sg.item_first;
      const bool whole = item_first >= share.c0 && item_first + item.steps <= share.c1;
      uint8_t* piece = static_cast<uint8_t*>(a.ws) + kAttnCounterBytes +
                       (size_t)(2 * blockIdx.x + (item_first < share.c0 ? 0 : 1)) * attn_piece_bytes(ROWS, D);
      named_barrier<128>(bar);
      if (t < 16 * hch) {
        const int j = hc + t;
        const float L = (wsum[0][j] + wsum[1][j]) + (wsum[2][j] + wsum[3][j]);
        if (!whole)
          reinterpret_cast<float2*>(piece + (size_t)ROWS * D * 4)[j] = make_float2(L > 0.f ? -neg_m[j] : kNoMax, L);
        sums[j] = L == 0.f ? 0.f : __frcp_rn(L);  // what the outputs are multiplied with
      }
      named_barrier<128>(bar);
      // ---- the segment's results ----
      const int g = gi + n - 1;
      if (wait_warp(o_done + (g & 1), (g >> 1) & 1)) {
        tc_after();
#pragma unroll 1
        for (int ch = 0; ch < hch; ++ch) {
          float o[16];
          tmem_ld16(t_o + 16 * ch, o);
          tmem_wait_ld(o);
          const int j0 = hc + 16 * ch;
          if (!whole) {
            float* dst = reinterpret_cast<float*>(piece) + j0 * D + t;
#pragma unroll
            for (int j = 0; j < 16; ++j) dst[j * D] = o[j];  // (rows past the item's are scratch)
          } else if (t < a.D) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int to = row_info[j0 + j].z;
              const float f = sums[j0 + j];
              if (to >= 0) a.out[(size_t)to * a.D + t] = (uint16_t)f32_to_bf16x2(f == 0.f ? 0.f : o[j] * f, 0.f);
            }
          }
        }
        tc_before();
      }
      if (u == 0 && item_first >= share.c0 && item_first + item.steps > share.c1) {
        // the item goes on in other shares: their pieces are joined by attn_kv8_join_kernel
        const int e = attn_cta_of<TcCut>(batch, share, item_first + item.steps - 1);
        split = make_int4((e - (int)blockIdx.x + 1) | rows << 16, sg.q0, item.h, item.rt);
      }
      named_barrier<256>(3);  // both halves are done with the tables of this segment
    }
    if (tid == 128) tc_splits(a.ws)[blockIdx.x] = abort_flag ? make_int4(0, 0, 0, 0) : split;
  }
  // After a wait that gave up: what is still in flight lands before the memory is given back (bounded waits).
  __syncthreads();
  if (abort_flag) {
    if (warp == 14 && lane == 0)
      for (int i = 0; i < stages; ++i)
        for (int ph = 0; ph < 2; ++ph) mbar_wait_n(full + i, ph, nullptr, 0, 1u << 14);
    if (warp == 15 && lane == 0) {
      tc_commit(o_done);
      for (int ph = 0; ph < 2; ++ph) mbar_wait_n(o_done, ph, nullptr, 0, 1u << 14);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 15) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTcCols));
  }
}

// Adds up the pieces of the items that go over several CTAs' shares, in the order
// of the CTAs. A unit is four rows of an item; the units are dealt over the grid.
// A row's 128 elements are a warp's, four warps share a row's pieces.
constexpr int kJoinRows = 4, kJoinParts = 4;
constexpr int kJoinThreads = 32 * kJoinRows * kJoinParts;
__global__ void __launch_bounds__(kJoinThreads) attn_kv8_join_kernel(AttnArgs a, int ctas) {
  __shared__ int4 items[kTcMaxCtas];  // .x: first CTA | rows << 16
  __shared__ int pieces_of[kTcMaxCtas], unit_end[kTcMaxCtas], found;
  __shared__ float4 part[kJoinParts][kJoinRows][32];
  __shared__ float2 stat[kJoinParts][kJoinRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.Hq / a.Hkv;
  const int row = warp % kJoinRows, mine = warp / kJoinRows;
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {  // the items that are in pieces, and their units' prefix sums
    int n = 0, units = 0;
    constexpr int kTimes = (kTcMaxCtas + 31) / 32;
    int4 all[kTimes];
#pragma unroll
    for (int k = 0; k < kTimes; ++k)
      all[k] = 32 * k + lane < ctas ? tc_splits(a.ws)[32 * k + lane] : make_int4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kTimes; ++k) {
      const int4 s = all[k];
      const int c0 = 32 * k;
      const bool in = (s.x & 0xFFFF) >= 2;
      const unsigned votes = __ballot_sync(0xffffffffu, in);
      int u = in ? ((s.x >> 16) + kJoinRows - 1) / kJoinRows : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, u, o);
        if (lane >= o) u += x;
      }
      if (in) {
        const int at = n + __popc(votes & ((1u << lane) - 1u));
        items[at] = make_int4((c0 + lane) | (s.x >> 16) << 16, s.y, s.z, s.w);
        pieces_of[at] = s.x & 0xFFFF;
        unit_end[at] = units + u;
      }
      n += __popc(votes);
      units += __shfl_sync(0xffffffffu, u, 31);
    }
    if (lane == 0) found = n;
  }
  __syncthreads();
  const int n = found;
  const uint8_t* ws = static_cast<const uint8_t*>(a.ws) + kAttnCounterBytes;
#pragma unroll 1
  for (int unit = blockIdx.x, it = 0; n > 0 && unit < unit_end[n - 1]; unit += gridDim.x) {
    while (unit >= unit_end[it]) ++it;
    const int4 item = items[it];
    const int first = item.x & 0xFFFF, rows = item.x >> 16, pieces = pieces_of[it];
    const int rr = (unit - (it > 0 ? unit_end[it - 1] : 0)) * kJoinRows + row;
    auto piece = [&](int i) {
      return ws + (size_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * attn_piece_bytes(kTcRows, D);
    };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kNoMax, l = 0.f;
    if (rr < rows) {
      // pieces mine, mine + 4, ..., eight on the way at a time, with a running maximum
#pragma unroll 1
      for (int i0 = mine; i0 < pieces; i0 += 8 * kJoinParts) {
        float2 st[8];
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = i0 + k * kJoinParts;
          if (i < pieces) {
            st[k] = __ldcg(reinterpret_cast<const float2*>(piece(i) + (size_t)kTcRows * D * 4) + rr);
            v[k] = __ldcg(reinterpret_cast<const float4*>(piece(i)) + rr * (D / 4) + lane);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (i0 + k * kJoinParts < pieces) {
            const float mn = fmaxf(m, st[k].x), f = ex2(m - mn), x = ex2(st[k].x - mn);
            m = mn;
            l = fmaf(st[k].y, x, l * f);
            o.x = fmaf(v[k].x, x, o.x * f), o.y = fmaf(v[k].y, x, o.y * f);
            o.z = fmaf(v[k].z, x, o.z * f), o.w = fmaf(v[k].w, x, o.w * f);
          }
        }
      }
    }
    part[mine][row][lane] = o;
    if (lane == 0) stat[mine][row] = make_float2(m, l);
    __syncthreads();
    if (mine == 0 && rr < rows && 4 * lane < a.D) {
      float mm = m;
#pragma unroll
      for (int p = 1; p < kJoinParts; ++p) mm = fmaxf(mm, stat[p][row].x);
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll
      for (int p = 0; p < kJoinParts; ++p) {
        const float2 st = stat[p][row];
        const float4 v = part[p][row][lane];
        const float x = ex2(st.x - mm);
        l = fmaf(st.y, x, l);
        o.x = fmaf(v.x, x, o.x), o.y = fmaf(v.y, x, o.y), o.z = fmaf(v.z, x, o.z), o.w = fmaf(v.w, x, o.w);
      }
      const float r = l == 0.f ? 0.f : __frcp_rn(l);
      const int rho = item.w * kTcRows + rr, qi = rho / G;
      const size_t to = (size_t)(item.y + qi) * a.Hq + item.z * G + rho - qi * G;
      *reinterpret_cast<uint2*>(a.out + to * a.D + 4 * lane) =
          make_uint2(f32_to_bf16x2(o.x * r, o.y * r), f32_to_bf16x2(o.z * r, o.w * r));
    }
    __syncthreads();
  }
}

template <int FMT>
cudaError_t launch_tc(const AttnArgs& a, cudaStream_t stream, bool pdl) {
  using S = TcShape;
  CUtensorMap km, vm;
  // tokens of a copy: the largest part of a step that lies in one block whatever its start
  const int box = a.bs % 128 == 0 ? 128 : a.bs % 64 == 0 ? 64 : a.bs % 32 == 0 ? 32 : 16;
  for (int i = 0; i < 2; ++i)
    if (!tmap_3d(i ? &vm : &km, CU_TENSOR_MAP_DATA_TYPE_UINT8, i ? a.v_cache : a.k_cache, a.D, a.bs,
                 (uint64_t)a.num_blocks * a.Hkv, a.D, (uint64_t)a.bs * a.D, D, box, 1))
      return cudaErrorInvalidValue;
  auto k = attn_kv8_tc_kernel<FMT>;
  cudaError_t e = allow_max_smem(k);
  if (e != cudaSuccess) return e;
  const size_t fixed = 2 * S::kV + 2 * S::kP + S::kQ + 16 * ((size_t)a.R + 1);
  // three stages; two where the tables of more than 800 requests leave no room
  const int stages = (int)std::min<size_t>(3, ((size_t)device_max_smem_optin() - 6144 - fixed) / S::kStage);
  const size_t smem = fixed + stages * S::kStage;
  const int ctas = std::min(device_sm_count(), kTcMaxCtas);
  e = launch_kernel(k, dim3(ctas), dim3(kTcThreads), smem, stream, pdl, km, vm, a, box, stages);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_kv8_join_kernel, dim3(ctas), dim3(kJoinThreads), 0, stream, true, a, ctas);
}

}  // namespace

cudaError_t launch_attn_kv8_tc(const AttnArgs& a, int format, cudaStream_t stream, bool pdl) {
  return format == QG_KV_I8 ? launch_tc<QG_KV_I8>(a, stream, pdl) : launch_tc<QG_KV_E4M3>(a, stream, pdl);
}

}  // namespace qg
