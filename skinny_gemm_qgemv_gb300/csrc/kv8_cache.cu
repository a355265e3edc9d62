// The paged 8-bit key/value cache: the block plan, the append and the read.
//
// kv8_plan_kernel. The lengths of all requests fit in one CTA's shared memory,
// so every CTA forms the prefix sums of the blocks taken, the blocks released
// and the new tokens by itself and then writes its share of the table, the
// stack and the slots. No CTA waits for another one's writes: a block taken at
// stack place p is free_list[p] below the old count, which nothing overwrites,
// and above it a block released in this call, found through the prefix sums in
// the releasing request's row, which nothing overwrites either. Few requests
// are one CTA and all latency (32: 4 us); 512 prompts of up to 4096 tokens,
// 6.7 MB written, take 8.8 us, 3 of them the scans.
//
// kv8_append_kernel. One CTA per window of tokens, head and cache (keys or values); it finds the runs that begin there.
// A run's maximum decides the block's scale, the earlier codes of the block are
// rounded to a grown scale, the run is quantized. All IEEE fp32 operations on
// single values, so the codes do not depend on the work's order. A run is read
// once (kept in registers between the maximum and the codes) and is a chain of
// slot map -> values -> maximum -> codes, so what bounds it is how many runs an SM
// holds: 4093 tokens of 8 heads of 128 from fp32, 33.5 MB, 12 us (2.8 TB/s).
//
// kv8_read_kernel. One CTA per block, head and cache, 8-byte loads and 16-byte
// stores: 8.4 MB of codes to 16.8 MB of bf16 in 5 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kPlanThreads = 512;

// take and rel are bounded by R * max_blocks < 2^31, the tokens only by their check
struct PlanSums {
  int take, rel;
  long long tok;
  int flags;  // joined, not summed
};

// exclusive prefix sums over the CTA; `total` gets the sums of all threads
__device__ __forceinline__ PlanSums plan_scan(PlanSums v, PlanSums* part, PlanSums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PlanSums s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, s.take, o), b = __shfl_up_sync(0xffffffffu, s.rel, o);
    const long long c = __shfl_up_sync(0xffffffffu, s.tok, o);
    if (lane >= o) s.take += a, s.rel += b, s.tok += c;
  }
  s.flags = __reduce_or_sync(0xffffffffu, v.flags);
  if (lane == 31) part[warp] = s;
  __syncthreads();
  PlanSums before = {0, 0, 0, 0};
  total = {0, 0, 0, 0};
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) before.take += part[w].take, before.rel += part[w].rel, before.tok += part[w].tok;
    total.take += part[w].take, total.rel += part[w].rel, total.tok += part[w].tok;
    total.flags |= part[w].flags;
  }
  return {before.take + s.take - v.take, before.rel + s.rel - v.rel, before.tok + s.tok - v.tok, 0};
}

// largest r in [0, n) with a[r] <= v, for ascending a with a[0] <= v
__device__ __forceinline__ int last_not_above(const int* a, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) kv8_plan_kernel(PlanArgs a) {
  extern __shared__ int sm[];
  int* take_ex = sm;                    // [R + 1] blocks taken before the request
  int* rel_ex = sm + a.R + 1;           // [R + 1] blocks released before it
  int* tok_ex = sm + 2 * (a.R + 1);     // [R + 1] new tokens before it
  int2* blocks = reinterpret_cast<int2*>(sm + (3 * a.R + 4) / 2 * 2);  // [R] blocks held before and after
  int* olds = reinterpret_cast<int*>(blocks + a.R);                    // [R]
  __shared__ PlanSums part[kPlanThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  const int per = (a.R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const int count = *a.free_count;
  PlanSums mine = {0, 0, 0, 0};  // flags 2: a request outgrows the table, 4: a negative length
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const int o = a.old_lens[r], n = a.new_lens[r];
    take_ex[r] = mine.take, rel_ex[r] = mine.rel, tok_ex[r] = (int)mine.tok;
    olds[r] = o;
    if (o < 0 || n < 0) {
      mine.flags |= 4;
    } else if (max(o, n) > a.max_blocks * a.bs) {
      mine.flags |= 2;
    } else {
      const int have = (o + a.bs - 1) / a.bs, need = (n + a.bs - 1) / a.bs;
      blocks[r] = make_int2(have, need);
      mine.take += max(0, need - have);
      mine.rel += max(0, have - need);
      mine.tok += max(0, n - o);
    }
  }
  PlanSums total;
  const PlanSums ex = plan_scan(mine, part, total);
  const int top = count + total.rel;
  int state = 0;
  if ((total.flags & 4) || count < 0 || count > a.num_blocks || total.rel > a.num_blocks - count)
    state = 4;
  else if (total.flags & 2)
    state = 2;
  else if (total.tok > a.max_tokens)
    state = 3;
  else if (total.take > top)
    state = 1;
  if (state) total = {0, 0, 0, 0};
#pragma unroll 1
  for (int r = r0; r < r1; ++r) take_ex[r] += ex.take, rel_ex[r] += ex.rel, tok_ex[r] += (int)ex.tok;
  if (tid == 0) take_ex[a.R] = total.take, rel_ex[a.R] = total.rel, tok_ex[a.R] = (int)total.tok;
  __syncthreads();
  // the block of rank j among those taken
  auto taken = [&](int j) {
    const int p = top - 1 - j;
    if (p < count) return a.free_list[p];
    const int r = last_not_above(rel_ex, a.R, j);  // also the rank among the released
    return a.table[(size_t)r * a.max_blocks + blocks[r].y + (j - rel_ex[r])];
  };
  // Three lists of independent writes, each begun at another thread, so that short ones run side by side.
  const int nthreads = gridDim.x * kPlanThreads, gid = blockIdx.x * kPlanThreads + tid;
  const int tokens = (int)total.tok;
#pragma unroll 1
  for (int t0 = 4 * gid; t0 < a.max_tokens; t0 += 4 * nthreads) {
    int slot[4], pos[4];
    // the request, its block and the place in it move on from token to token
    int r = -1, p = 0, end = t0, blk = 0, b = 0, off = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i;
      slot[i] = pos[i] = -1;
      if (t < tokens) {
        bool look = off == a.bs;
        if (t >= end) {
          if (r < 0)
            r = last_not_above(tok_ex, a.R, t);
          else
            while (tok_ex[r + 1] <= t) ++r;
          end = tok_ex[r + 1];
          p = olds[r] + t - tok_ex[r];
          b = p / a.bs;
          off = p - b * a.bs;
          look = true;
        } else if (look) {
          ++b;
          off = 0;
        }
        if (look) {
          const int have = blocks[r].x;
          blk = b < have ? a.table[(size_t)r * a.max_blocks + b] : taken(take_ex[r] + b - have);
        }
        slot[i] = blk * a.bs + off;
        pos[i] = p;
        ++off, ++p;
      }
    }
    if (t0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (t0 + i < a.max_tokens) a.slot_map[t0 + i] = slot[i], a.positions[t0 + i] = pos[i];
      }
    }
  }
  const int gid_take = gid >= nthreads / 2 ? gid - nthreads / 2 : gid + (nthreads - nthreads / 2);
#pragma unroll 1
  for (int j = gid_take; j < total.take; j += nthreads) {
    const int r = last_not_above(take_ex, a.R, j);
    a.table[(size_t)r * a.max_blocks + blocks[r].x + (j - take_ex[r])] = taken(j);
  }
  const int gid_rel = gid >= nthreads / 4 * 3 ? gid - nthreads / 4 * 3 : gid + (nthreads - nthreads / 4 * 3);
#pragma unroll 1
  for (int k = gid_rel; k < total.rel; k += nthreads) {
    const int r = last_not_above(rel_ex, a.R, k);
    a.free_list[top - 1 - k] = a.table[(size_t)r * a.max_blocks + blocks[r].y + (k - rel_ex[r])];
  }
  if (blockIdx.x == gridDim.x - 1) {
#pragma unroll 1
    for (int r = tid; r <= a.R; r += kPlanThreads) a.cu_new[r] = state ? 0 : tok_ex[r];
    if (tid == 0) *reinterpret_cast<int4*>(a.info) = make_int4(tokens, total.take, total.rel, state);
  }
  // free_count_out may be free_count: the CTA that read it last writes it (no one waits)
  if (tid == 0) {
    const int left = state ? count : top - total.take;
    if (gridDim.x == 1) {
      *a.free_count_out = left;
    } else {
      unsigned seen;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(seen) : "l"(a.ticket) : "memory");
      if (seen == gridDim.x - 1) {
        *a.free_count_out = left;
        *a.ticket = 0;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

__device__ __forceinline__ void load8_in(const void* p, int f32, size_t elem, float (&v)[8]) {
  if (f32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + elem);
    const float4 a = __ldcs(s), b = __ldcs(s + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + elem));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

// KEEP: steps of 8 elements that a thread keeps between the maximum and the codes (what is more is read again)
template <int FMT, int THREADS, int KEEP>
__global__ void __launch_bounds__(THREADS, KEEP == 1 ? 2048 / THREADS : KEEP == 2 ? 1280 / THREADS : 1024 / THREADS) kv8_append_kernel(AppendArgs a) {
  __shared__ int lead[THREADS], leads;
  __shared__ int part_n[THREADS / 32];
  __shared__ float part[THREADS / 32];
  const int tid = threadIdx.x;
  if (tid == 0) leads = 0;
  pdl_wait();
  pdl_launch_dependents();
  const int which = blockIdx.y & 1, head = blockIdx.y >> 1;
  const void* x = which ? a.v : a.k;
  const long long stride = which ? a.v_stride : a.k_stride;
  uint8_t* cache = static_cast<uint8_t*>(which ? a.v_cache : a.k_cache);
  const int d8 = a.D / 8;
  __syncthreads();
  {
    // the first tokens of runs in this CTA's window (slots of a block ascend by one)
    const int t = blockIdx.x * a.window + tid;
    if (tid < a.window && t < a.T) {
      const int slot = a.slot_map[t], prev = t > 0 ? a.slot_map[t - 1] : -1;
      if (slot >= a.num_blocks * a.bs)
        report_error(a.err, kErrKvSlot);
      else if (slot >= 0 && (slot % a.bs == 0 || prev != slot - 1))
        lead[atomicAdd(&leads, 1)] = t;
    }
  }
  __syncthreads();
  for (int k = 0; k < leads; ++k) {
    const int t0 = lead[k], slot = a.slot_map[t0], f = slot % a.bs, blk = slot / a.bs;
    // The run's length: up to the block's end or the first slot that does not follow. The values it can have are
    // loaded before it is known.
    const int most = min(a.bs - f, a.T - t0);
    auto at = [&](int i) { return (t0 + i / d8) * stride + head * a.D + (i % d8) * 8; };
    float keep[KEEP][8];
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
      const int i = tid + c * THREADS;
      if (i < most * d8) load8_in(x, a.f32, at(i), keep[c]);
    }
    int n = most;
    for (int i = tid; i < most; i += THREADS)
      if (a.slot_map[t0 + i] != slot + i) n = min(n, i);
    n = __reduce_min_sync(0xffffffffu, n);
    if ((tid & 31) == 0) part_n[tid >> 5] = n;
    float* sp = a.scales + 2 * ((size_t)blk * a.Hkv + head) + which;
    const float s0 = f > 0 ? *sp : 0.f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) n = min(n, part_n[w]);
    const int chunks = n * d8;
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
      if (tid + c * THREADS < chunks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(keep[c][j]));
      }
    }
    for (int i = tid + KEEP * THREADS; i < chunks; i += THREADS) {
      float v[8];
      load8_in(x, a.f32, at(i), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) part[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, part[w]);
    const float s = fmaxf(s0, __fdiv_rn(amax, kv8_qmax<FMT>()));
    if (tid == 0) *sp = s;  // every thread read the old one before the barrier
    uint8_t* page = cache + ((size_t)blk * a.Hkv + head) * a.bs * a.D;
    if (f > 0 && s > s0) {
      // the earlier codes, rounded to the grown scale
      const float ratio = __fdiv_rn(s0, s);
      for (int i = tid; i < f * d8; i += THREADS) {
        uint2* p = reinterpret_cast<uint2*>(page) + i;
        const uint2 old = *p;
        float v[8];
        kv8_decode4<FMT>(old.x, v[0], v[1], v[2], v[3]);
        kv8_decode4<FMT>(old.y, v[4], v[5], v[6], v[7]);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], ratio);
        *p = make_uint2(kv8_encode4<FMT>(v[0], v[1], v[2], v[3]), kv8_encode4<FMT>(v[4], v[5], v[6], v[7]));
      }
    }
    uint2* dst = reinterpret_cast<uint2*>(page + (size_t)f * a.D);
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int c = 0; c < KEEP; ++c) {
      const int i = tid + c * THREADS;
      if (i < chunks) dst[i] = s > 0.f ? kv8_quantize8<FMT>(keep[c], s, inv) : make_uint2(0u, 0u);
    }
    for (int i = tid + KEEP * THREADS; i < chunks; i += THREADS) {
      float v[8];
      load8_in(x, a.f32, at(i), v);
      dst[i] = s > 0.f ? kv8_quantize8<FMT>(v, s, inv) : make_uint2(0u, 0u);
    }
    if (f == 0)
      for (int i = tid + chunks; i < a.bs * d8; i += THREADS) dst[i] = make_uint2(0u, 0u);
    // (part_n and part are written again only after a barrier that follows their last reads)
  }
}

// ---------------------------------------------------------------------------
// read
// ---------------------------------------------------------------------------
template <int FMT>
__global__ void __launch_bounds__(256) kv8_read_kernel(ReadArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int which = blockIdx.z, head = blockIdx.y;
  const int per = a.bs * a.D / 8;
  const int id = a.ids[blockIdx.x];
  const bool ok = id >= 0 && id < a.num_blocks;
  if (!ok && threadIdx.x == 0) report_error(a.err, kErrKvBlock);
  const size_t page = ((size_t)(ok ? id : 0) * a.Hkv + head);
  const size_t dst = ((size_t)blockIdx.x * a.Hkv + head);
  const float s = ok ? a.scales[2 * page + which] : 0.f;
  if (threadIdx.x == 0) a.scales_out[2 * dst + which] = s;
  const uint2* src = reinterpret_cast<const uint2*>(which ? a.v_cache : a.k_cache) + page * per;
  uint4* out = reinterpret_cast<uint4*>(which ? a.v : a.k) + dst * per;
  for (int i = threadIdx.x; i < per; i += blockDim.x) {
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (ok) {
      const uint2 c = src[i];
      float v[8];
      kv8_decode4<FMT>(c.x, v[0], v[1], v[2], v[3]);
      kv8_decode4<FMT>(c.y, v[4], v[5], v[6], v[7]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      o = make_uint4(f32_to_bf16x2(v[0], v[1]), f32_to_bf16x2(v[2], v[3]), f32_to_bf16x2(v[4], v[5]),
                     f32_to_bf16x2(v[6], v[7]));
    }
    out[i] = o;
  }
}

}  // namespace

cudaError_t launch_kv8_plan(const PlanArgs& a, cudaStream_t stream, bool pdl) {
  // four tokens a thread; each CTA forms the sums anew (a few us, side by side)
  const int ctas =
      std::min(4 * device_sm_count(), std::max(1, (a.max_tokens + 4 * kPlanThreads - 1) / (4 * kPlanThreads)));
  const size_t smem = sizeof(int) * (6 * (size_t)a.R + 8);
  if (smem > 40 << 10) {
    cudaError_t e = allow_max_smem(kv8_plan_kernel);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kv8_plan_kernel, dim3(ctas), dim3(kPlanThreads), smem, stream, pdl, a);
}

cudaError_t launch_kv8_append(AppendArgs a, int format, cudaStream_t stream, bool pdl) {
  // Tokens whose runs one CTA takes: one where that gives up to eight CTAs an SM, up to a block of them (and no more
  // than a CTA has threads) for a long prompt.
  a.window = (int)std::min<long long>(std::min(a.bs, 128),
                                      std::max<long long>(1, (long long)a.T * a.Hkv * 2 / (8 * device_sm_count())));
  const dim3 grid((a.T + a.window - 1) / a.window, 2 * a.Hkv);
  auto launch = [&](auto i8, auto e4m3, int threads) {
    return launch_kernel(format == QG_KV_I8 ? i8 : e4m3, grid, dim3(threads), 0, stream, pdl, a);
  };
  // By the elements of a run: no more registers and threads than it needs, for the more runs are on the way per SM.
  // With the read-back, 4093 tokens of 8 heads of 128: blocks of 16 30.0 us in the widest form, 22.4 with 256 threads and
  // one step, 21.2 as here; blocks of 32 23.2 and 20.1; blocks of 64 (fp32) 16.5, 19.4 with 512 threads.
  const int elems = a.bs * a.D;
  if (elems <= 1024) return launch(kv8_append_kernel<QG_KV_I8, 128, 1>, kv8_append_kernel<QG_KV_E4M3, 128, 1>, 128);
  if (elems <= 2048) return launch(kv8_append_kernel<QG_KV_I8, 128, 2>, kv8_append_kernel<QG_KV_E4M3, 128, 2>, 128);
  if (elems <= 4096) return launch(kv8_append_kernel<QG_KV_I8, 256, 2>, kv8_append_kernel<QG_KV_E4M3, 256, 2>, 256);
  return launch(kv8_append_kernel<QG_KV_I8, 256, 4>, kv8_append_kernel<QG_KV_E4M3, 256, 4>, 256);
}

cudaError_t launch_kv8_read(const ReadArgs& a, int format, cudaStream_t stream, bool pdl) {
  auto k = format == QG_KV_I8 ? kv8_read_kernel<QG_KV_I8> : kv8_read_kernel<QG_KV_E4M3>;
  return launch_kernel(k, dim3(a.B, a.Hkv, 2), dim3(256), 0, stream, pdl, a);
}

}  // namespace qg
