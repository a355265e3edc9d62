// A token per row of logits, drawn from the softmax cut by temperature, top-k,
// top-p and min-p, with one given random number a row.
//
// The tokens of a row in descending order of their logits (the lower index first
// among equal ones) have weights w_j = exp((x_j - x_max) / T) and sums C_n = w_1 + ..
// + w_n. What is kept is always a beginning of that order: the k first, then the
// fewest n with C_n >= p C_k, then those with x - x_max >= T ln(min_p). The token is
// the first one with C_i > u C_n.
//
// No row is sorted. A cluster of CTAs holds the row in its shared memory (a bulk
// copy each: HBM is read once), takes the maximum, and counts the tokens in 2047
// bins of equal width below it; what a cut or the draw needs of the order lies in
// one bin, or for small cuts in the first few: those tokens alone are gathered and
// sorted by one CTA. For cuts that keep a few hundred tokens a sample tells where
// they begin, and nothing is counted.
//
// Weights are whole numbers, in units of 2^-43 of the largest one: the weight of the
// middle of the token's bin less its deviation from that, which is a multiple of a
// power of two that the bin has (half of it is at most 2^-22 of the weight). A bin's
// sum is then its count times its middle's weight less the sum of its tokens'
// deviations, by 32-bit atomics in shared memory, and the same to the last digit as
// the sum of its tokens' weights one by one: neither an order of atomics or threads
// nor the way by which a row's token is found changes a result. Distances from the
// maximum are formed without error from two fp32.
//
// Measured (fp32 logits unless said): one row of 151936 13 us, 32 rows 18 to 20, each some twenty phases between barriers of
// a cluster, of 500 to 5000 cycles (a warp issues in one of 18; code that runs once a row is slow to fetch too); 61 bf16
// rows of 50021 without top-k 34 to 36, the slowest of which try a list, count all tokens and gather two bins; 512 rows of
// 151936 drawn from the whole softmax 250 (46 us for the bytes): four waves of rows, each 16 us for the maximum and 15 for
// the list at the copy rate and 33 for the count, whose two shared atomics a token bound it. Rows that are searched by
// halving: one of equal logits 0.4 ms, 152 of them 2.5.
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

typedef unsigned long long u64;

constexpr int kBins = 2048;     // the last one takes what lies below the others
constexpr int kOver = kBins - 1;
constexpr int kList = 1024;     // tokens that are gathered and sorted, at most
constexpr int kFewK = 768;      // top-k up to which the bins only count
constexpr float kFewScale = 90.f;      // their number per unit of a logit
constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: leaves the nearest whole number in the low bits of a sum
constexpr int kMaxCluster = 8;

struct Found {  // a bin: the tokens and the weight before it, the tokens in it, the weight up to its end
  int bin, n, count, pad;
  u64 mass, after;
};
struct Row {  // what the CTAs of a cluster tell one another
  float max[kMaxCluster];
  int lowest[kMaxCluster];
  int count[kMaxCluster], listed[kMaxCluster], landed[kMaxCluster], over;
  float bound[kMaxCluster], below[kMaxCluster];
  int done;
  u64 mass[kMaxCluster], tail[kMaxCluster], sum[2][kMaxCluster];
  Found found[2];    // of two searches in turn
  u64 result[2];  // of a walk through a sorted list: the sum at its end, the place
};

__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void put32(const void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void put64(const void* p, int rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get32(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ u64 get64(const void* p, int rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr(p, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// fp32 as unsigned numbers of the same order; -0 is 0
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <class T, class OP>
__device__ __forceinline__ T warp_all(T v, OP op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// over the CTA, for all threads; `part` [warps] is free again after the caller's next barrier
template <int WARPS, class T, class OP>
__device__ __forceinline__ T cta_all_of(T v, OP op, T* part) {
  v = warp_all(v, op);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) v = op(v, part[w]);
  return v;
}
struct Add {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct Min {
  __device__ int operator()(int a, int b) const { return min(a, b); }
};

// The weight of a distance from the maximum, as described above: bins of 1 / S octaves, S = 64 << sj.
struct Scale {
  float max, ch, cl;  // ch + cl = S log2(e) / T
  float per;          // ln 2 / S
  float inv;          // -1 / S
  float end;          // bins from here on, 45 octaves down, weigh less than half a unit
  int sj;
};
__device__ __forceinline__ int bin_of(float a, float c) {
  return __float_as_int(fminf(a * c, (float)kOver) + kMagic) & 0xFFF;
}
// 1 - 2^(-r / S) for the distance of a from the middle of bin b, |r| <= 1/2 or little more
__device__ __forceinline__ float deviation(const Scale& s, float x, float a, float b) {
  const float t = a - s.max, e = (s.max - (a - t)) + (-x - t);  // a + e = max - x
  const float r = fmaf(a, s.ch, -b) + fmaf(a, s.cl, e * s.ch), y = r * s.per;
  return y * fmaf(y, fmaf(y, 1.f / 6.f, -0.5f), 1.f);
}
// 2^(-i / 64) and 2^(-i / 4096), i = 0 .. 63, in units of 2^-63, rounded to nearest
__constant__ u64 kPow[2][64] = {
    {
     0x8000000000000000ull, 0x7e9f06067a4360baull, 0x7d41d96db915019dull, 0x7be86fb985689ddcull,
     0x7a92be8a92436616ull, 0x7940bb9e2cffd89dull, 0x77f25ccdee6d7ae6ull, 0x76a7980f6cca15c2ull,
     0x75606373ee921c97ull, 0x741cb5281e25ee34ull, 0x72dc8373be41a454ull, 0x719fc4b95f452d29ull,
     0x70666f76154a7089ull, 0x6f307a412f074892ull, 0x6dfddbcbed791babull, 0x6cce8ae13c57ebdbull,
     0x6ba27e656b4eb57aull, 0x6a79ad55e7f6fd10ull, 0x69540ec8f895722dull, 0x683199ed779592caull,
     0x6712460a8fc24072ull, 0x65f60a7f79393e2eull, 0x64dcdec3371793d1ull, 0x63c6ba6455dcd8aeull,
     0x62b39508aa836d6full, 0x61a3666d124bb204ull, 0x6096266533384a2bull, 0x5f8bccdb3d398841ull,
     0x5e8451cfac061b5full, 0x5d7fad59099f22feull, 0x5c7dd7a3b17dcf75ull, 0x5b7ec8f19468bbc9ull,
     0x5a827999fcef3242ull, 0x5988e20954889245ull, 0x5891fac0e95612c8ull, 0x579dbc56b48521baull,
     0x56ac1f752150a563ull, 0x55bd1cdad49f699cull, 0x54d0ad5a753e077cull, 0x53e6c9da74b29ab5ull,
     0x52ff6b54d8a89c75ull, 0x521a8ad704f3404full, 0x513821818624b40cull, 0x50582887dcb8a7e1ull,
     0x4f7a993048d088d7ull, 0x4e9f6cd3967fdba8ull, 0x4dc69cdceaa72a9cull, 0x4cf022c9905bfd32ull,
     0x4c1bf828c6dc54b8ull, 0x4b4a169b900c2d00ull, 0x4a7a77d47f7b84b1ull, 0x49ad159789f37496ull,
     0x48e1e9b9d588e19bull, 0x4818ee218a3358eeull, 0x47521cc5a2e6a9e0ull, 0x468d6fadbf2dd4f3ull,
     0x45cae0f1f545eb73ull, 0x450a6abaa4b77ecdull, 0x444c0740496d4294ull, 0x438fb0cb4f468808ull,
     0x42d561b3e6243d8aull, 0x421d1461d66f2023ull, 0x4166c34c5615d0ecull, 0x40b268f9de0183baull,
    },
    {
     0x8000000000000000ull, 0x7ffa748dff8dc61full, 0x7ff4e9597bed93abull, 0x7fef5e6272758c21ull,
     0x7fe9d3a8e07bf086ull, 0x7fe4492cc3571f68ull, 0x7fdebeee185d94ddull, 0x7fd934ecdce5ea7dull,
     0x7fd3ab290e46d769ull, 0x7fce21a2a9d73041ull, 0x7fc89859acede72aull, 0x7fc30f4e14e20bc6ull,
     0x7fbd867fdf0acb3bull, 0x7fb7fdef08bf7027ull, 0x7fb2759b8f5762aaull, 0x7faced85702a285dull,
     0x7fa765aca88f6453ull, 0x7fa1de1135ded717ull, 0x7f9c56b315705eaeull, 0x7f96cf92449bf692ull,
     0x7f9148aec0b9b7b1ull, 0x7f8bc2088721d86full, 0x7f863b9f952caca0ull, 0x7f80b573e832a58bull,
     0x7f7b2f857d8c51e5ull, 0x7f75a9d452925dd4ull, 0x7f702460649d92eaull, 0x7f6a9f29b106d825ull,
     0x7f651a30352731eeull, 0x7f5f9573ee57c218ull, 0x7f5a10f4d9f1c7ddull, 0x7f548cb2f54e9fdfull,
     0x7f4f08ae3dc7c426ull, 0x7f4984e6b0b6cc1dull, 0x7f44015c4b756c94ull, 0x7f3e7e0f0b5d77bcull,
     0x7f38fafeedc8dd26ull, 0x7f33782bf011a9c2ull, 0x7f2df5960f9207e1ull, 0x7f28733d49a43f2dull,
     0x7f22f1219ba2b4aeull, 0x7f1d6f4302e7eac6ull, 0x7f17eda17cce812eull, 0x7f126c3d06b134faull,
     0x7f0ceb159deae091ull, 0x7f076a2b3fd67bb2ull, 0x7f01e97de9cf1b6eull, 0x7efc690d992ff22aull,
     0x7ef6e8da4b544f9aull, 0x7ef168e3fd97a0c6ull, 0x7eebe92aad557001ull, 0x7ee669ae57e964edull,
     0x7ee0ea6efaaf4479ull, 0x7edb6b6c9302f0dfull, 0x7ed5eca71e4069a1ull, 0x7ed06e1e99c3cb8bull,
     0x7ecaefd302e950afull, 0x7ec571c4570d5067ull, 0x7ebff3f2938c3f4full, 0x7eba765db5c2af49ull,
     0x7eb4f905bb0d4f78ull, 0x7eaf7beaa0c8ec3eull, 0x7ea9ff0c64526f40ull, 0x7ea4826b0306df5full,
    },
};
// f z for an fp32 f in [0, 1), rounded up or down: exact (64-bit floating-point instructions, of which GB300 issues two
// lanes a cycle and SM, would take longer than the sweeps)
__device__ __forceinline__ u64 times(float f, u64 z, bool up) {
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const u64 m = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;  // f = m 2^-shift
  const int shift = 150 - (e ? (int)e : 1);                            // 24 or more
  const u64 lo = z * m, hi = __umul64hi(z, m);
  if (shift >= 88) return up && (lo | hi);
  const u64 whole = shift >= 64 ? hi >> (shift - 64) : hi << (64 - shift) | lo >> shift;
  const bool left = shift >= 64 ? (hi & ((1ull << (shift - 64)) - 1)) | lo : lo & ((1ull << shift) - 1);
  return whole + (up && left);
}
// 2^(-b / S) in units of 2^-63 for bins below the octave, and the octave
__device__ __forceinline__ u64 mantissa(const u64 (*pow)[64], int b, int sj) {
  return __umul64hi(pow[0][b >> sj & 63], pow[1][(b & ((1 << sj) - 1)) << (6 - sj)]) << 1;
}
// The middle of bin b (a whole number) as fp32, units of 2^-43; and as the factor of a deviation in that bin's steps of
// 2^shift units: from 2^(21 + sj) up to, but not, twice that where the middle is so large (deviations are then below 22780
// steps, whatever sj), and the middle itself, with steps of a unit, where it is less.
__device__ __forceinline__ float middle_f32(const Scale& s, float b) { return ex2(fmaf(b, s.inv, 43.f)); }
__device__ __forceinline__ float steps_of(const Scale& s, float middle, int& shift) {
  const uint32_t bits = __float_as_uint(middle), top = (uint32_t)(127 + 21 + s.sj) << 23, e = bits & 0x7F800000u;
  const uint32_t over = e - min(e, top);
  shift = (int)(over >> 23);
  return __uint_as_float(bits - over);
}
// the middle in whole units: small ones from fp32, off by less than one unit
__device__ __forceinline__ u64 middle_of(const u64 (*pow)[64], float middle, int b, int sj) {
  if (middle < 2097152.f) return (u64)__float2uint_rn(middle);
  return ((mantissa(pow, b, sj) >> (19 + (b >> (6 + sj)))) + 1) >> 1;
}
// steps by which x at distance a, of bin b and its factor, weighs less than the bin's middle
__device__ __forceinline__ int steps_below(const Scale& s, float x, float a, float b, float factor) {
  return __float_as_int(fmaf(deviation(s, x, a, b), factor, kMagic)) - 0x4B400000;
}
// The weight below the bins, th bins down. With S = 64 that is less than 2^11 units, and fp32 gives them to 2^-8 of one.
__device__ __forceinline__ uint32_t weight_below(const Scale& s, float th) {
  return __float_as_uint(ex2(fmaf(th, s.inv, 43.f)) + kMagic) - 0x4B400000u;
}
__device__ __forceinline__ u64 weight_of(const Scale& s, const u64 (*pow)[64], float x) {
  const float a = s.max - x, th = a * s.ch;
  if (!(th < s.end)) return 0ull;
  const float b = rintf(th), middle = middle_f32(s, b);
  if (s.sj == 0 && b >= (float)kOver) return weight_below(s, th);
  int shift;
  const float factor = steps_of(s, middle, shift);
  return middle_of(pow, middle, (int)b, s.sj) - (u64)(steps_below(s, x, a, b, factor) * (1ll << shift));
}

// weight_of / total as fp32, whatever the weight is
__device__ __forceinline__ float share_of(const Scale& s, const u64 (*pow)[64], float x, u64 total) {
  const float a = s.max - x, th = a * s.ch;
  if (!(th < 1048576.f)) return 0.f;
  const float bf = rintf(th);
  const int b = (int)bf, octave = b >> (6 + s.sj);
  const u64 w = __umul64hi(mantissa(pow, b, s.sj), (u64)((1ll << 44) - (long long)(deviation(s, x, a, bf) * 17592186044416.f)));
  return octave > 200 ? 0.f : (float)((double)w / (double)total * __hiloint2double((1023 - octave) << 20, 0));
}

// four consecutive elements
template <bool F32>
__device__ __forceinline__ void quad(const uint8_t* slice, int i, float (&x)[4]) {
  if (F32) {
    const float4 v = reinterpret_cast<const float4*>(slice)[i];
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const uint2 v = reinterpret_cast<const uint2*>(slice)[i];
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
}

// HELD: a cluster per row, which it holds in shared memory; else a CTA per row, which reads it again from L2 in every
// sweep
template <bool F32, bool HELD, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) sample_kernel(SampleArgs a, int cluster) {
  constexpr int PER = F32 ? 4 : 8;  // elements of 16 bytes
  constexpr int kWarps = kThreads / 32, kPlaces = kList / kThreads;  // places of a list that a thread has
  auto cta_all = [](auto v, auto op, auto* part) { return cta_all_of<kWarps>(v, op, part); };
  extern __shared__ __align__(16) uint8_t smem[];
  // layout: bins' counts | their deviations (| both again, of the warps of odd number) | sums before this CTA's bins |
  // tokens before them | the slice
  constexpr int kCopies = HELD ? 1 : 2;
  int* cnt = reinterpret_cast<int*>(smem);
  int* dev = cnt + kBins;
  const int own_bins = HELD ? kBins / cluster : kBins;
  u64* before_m = reinterpret_cast<u64*>(cnt + 2 * kCopies * kBins);
  int* before_n = reinterpret_cast<int*>(before_m + own_bins);
  uint8_t* slice = reinterpret_cast<uint8_t*>(before_n + own_bins);
  // a gathered list over the counts, its sorted whole (in CTA 0) over the deviations
  u64* list = reinterpret_cast<u64*>(cnt);
  u64* sorted = reinterpret_cast<u64*>(dev);
  __shared__ Row row;
  __shared__ u64 pow[2][64];
  __shared__ __align__(16) u64 splitter[32];  // of a sort
  __shared__ int part_size[33], part_begin[34];
  __shared__ uint8_t part_of[kList];
  __shared__ u64 part64[kWarps];
  __shared__ int part32[kWarps];
  __shared__ float partf[kWarps], part_below[kWarps];
  __shared__ uint64_t bar;
  __shared__ int taken;
  __shared__ u64 tail_of;           // what lies below the bins
  __shared__ float step_of[2];      // the scale's ch, cl
  __shared__ double least_of;       // T ln(min_p)
  __shared__ float least_at;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = HELD ? blockIdx.x / cluster : blockIdx.x, rank = HELD ? blockIdx.x % cluster : 0;
  if (!HELD) cluster = 1;
  int* my_cnt = cnt + (HELD ? 0 : (warp & 1) * 2 * kBins);
  int* my_dev = my_cnt + kBins;
  const int size = F32 ? 4 : 2;

  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  if (tid < 128) pow[tid >> 6][tid & 63] = kPow[tid >> 6][tid & 63];
  if (HELD) cluster_arrive();  // every CTA of the cluster runs once this is through: its memory may be written
  // of the cluster, or of the CTA alone
  auto all_sync = [&]() {
    if (HELD)
      cluster_sync();
    else
      __syncthreads();
  };
  auto tell32 = [&](const void* at, int r, uint32_t v) {
    if (HELD)
      put32(at, r, v);
    else
      *reinterpret_cast<volatile uint32_t*>(const_cast<void*>(at)) = v;
  };
  auto tell64 = [&](const void* at, int r, u64 v) {
    if (HELD)
      put64(at, r, v);
    else
      *reinterpret_cast<volatile u64*>(const_cast<void*>(at)) = v;
  };
  auto ask32 = [&](const void* at, int r) { return HELD ? get32(at, r) : *static_cast<const uint32_t*>(at); };
  auto ask64 = [&](const void* at, int r) { return HELD ? get64(at, r) : *static_cast<const u64*>(at); };
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();

  // ---- the slice: 16-byte units of the row from its first 16-byte boundary on; what lies before that and after the last
  // whole unit fills up a unit of the first and of the last CTA, with -infinity around it
  const char* base = static_cast<const char*>(a.logits) + m * a.stride * size;
  const int head = (int)((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / size;
  const int lead = min(head, a.V), units = (a.V - lead) / PER, rest = a.V - lead - units * PER;
  const int u0 = (int)((long long)units * rank / cluster), u1 = (int)((long long)units * (rank + 1) / cluster);
  const int front = rank == 0 && lead ? 1 : 0, back = rank == cluster - 1 && rest ? 1 : 0;
  const int n = front + (u1 - u0) + back;                    // units in shared memory
  const int first = lead + (u0 - front) * PER;               // index of the first one's first element
  if (HELD && tid == 0) {
    const uint32_t bytes = (uint32_t)(u1 - u0) * 16u;
    mbar_arrive_expect_tx(&bar, bytes);
    constexpr uint32_t kPiece = 32768u;
    const char* src = base + (size_t)(lead + u0 * PER) * size;
#pragma unroll 1
    for (uint32_t at = 0; at < bytes; at += kPiece)
      bulk_g2s(slice + 16 * front + at, src + at, min(kPiece, bytes - at), &bar);
  }
  if (HELD && tid < 2 * PER) {
    const int j = tid % PER, which = tid / PER;               // 0: the front unit, 1: the back one
    const int e = which ? lead + units * PER + j : lead - PER + j;
    const bool in = which ? j < rest : e >= 0;
    if (which ? back : front) {
      uint8_t* to = which ? slice + 16 * (n - 1) : slice;
      if (F32)
        reinterpret_cast<uint32_t*>(to)[j] = in ? reinterpret_cast<const uint32_t*>(base)[e] : 0xFF800000u;
      else
        reinterpret_cast<uint16_t*>(to)[j] = in ? reinterpret_cast<const uint16_t*>(base)[e] : (uint16_t)0xFF80u;
    }
  }
  const float u_raw = a.u[m];
  const float u = u_raw >= 0.f ? fminf(u_raw, 0.99999994f) : 0.f;
  const float temp = a.temperature ? a.temperature[m] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float T = fminf(fmaxf(temp, 1e-30f), 1e30f);
  long long k_raw = 0;
  if (a.top_k) k_raw = a.k64 ? static_cast<const long long*>(a.top_k)[m] : static_cast<const int*>(a.top_k)[m];
  const float p_raw = a.top_p ? a.top_p[m] : 1.f, mp_raw = a.min_p ? a.min_p[m] : 0.f;
  const int k = k_raw > 0 && k_raw < a.V ? (int)k_raw : 0;   // 0: all
  const bool has_p = p_raw < 1.f, has_m = mp_raw > 0.f;
  // The bins reach 22 T / 2^sj logits below the maximum: 22 at least, so that they hold the bulk below a high head too (with
  // 11, 512 rows of 151936 at temperatures of 0.6 to 1.2 and top-p took 2.4 ms instead of 0.31, searched by halving). Where
  // a bin of that width, 0.0108 T / 2^sj logits, would hold more tokens of a broad row than a list, they have half of it
  // (152 broad rows of 262144 at a temperature of 1.4 0.86 and 0.26 ms).
  int sj = 0;
  while (sj < 6 && T >= (float)(2 << sj)) ++sj;
  if (sj < 6 && T > (float)(1 << sj) && (float)a.V * T > 350000.f * (float)(1 << sj)) ++sj;
  // (by one warp: GB300 has two lanes an SM for 64-bit floating point)
  if (warp == 1 && !greedy) {
    const double c = 1.4426950408889634 * (64 << sj) / (double)T, at = has_m ? (double)T * log((double)fminf(mp_raw, 1.f)) : 0.;
    if (lane == 0) step_of[0] = (float)c, step_of[1] = (float)(c - (double)(float)c), least_of = at;
  }
  __syncthreads();
  bool landed = !HELD || __syncthreads_and(mbar_wait(&bar, 0, a.err, kErrSampleWait));

  constexpr float kMost = 3.402823466e+38f;
  const float largest = F32 ? kMost : __uint_as_float(0x7F7F0000u);
  const int quads = n * (PER / 4);
  auto index_of = [&](int i, int j) { return first + 4 * i + j; };
  bool clean = true;  // no logit is NaN or +infinity, as far as is known
  auto load = [&](int i, float (&x)[4]) {
    if (HELD) {
      quad<F32>(slice, i, x);
      return;
    }
    const int e = first + 4 * i;
    if (e >= 0 && e + 4 <= a.V) {
      quad<F32>(reinterpret_cast<const uint8_t*>(base) + (long long)e * size, 0, x);
    } else {
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        float v = -INFINITY;
        if (e + j >= 0 && e + j < a.V)
          v = F32 ? reinterpret_cast<const float*>(base)[e + j] : bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(base)[e + j]);
        x[0] = j == 0 ? v : x[0], x[1] = j == 1 ? v : x[1], x[2] = j == 2 ? v : x[2], x[3] = j == 3 ? v : x[3];
      }
    }
    if (clean) return;  // (the same for all threads)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = fminf(fmaxf(x[j], -INFINITY), largest);
  };
  // f(x, i, j) of element j of quad i, of all of the thread's. Held rows: no further unrolled (much of this code runs once
  // a row, and a short row's time is that of fetching it); others: four loads on the way. `slow`: what rarely runs.
  auto sweep_slow = [&](auto&& f) {
#pragma unroll 1
    for (int i = tid; i < quads; i += kThreads) {
      float x[4];
      load(i, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f(x[j], i, j);
    }
  };
  auto sweep = [&](auto&& f) {
    if (HELD) {
      sweep_slow(f);
      return;
    }
    constexpr int kDeep = 4;
    int i = tid;
#pragma unroll 1
    for (; i + (kDeep - 1) * kThreads < quads; i += kDeep * kThreads) {
      float x[kDeep][4];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) load(i + k * kThreads, x[k]);
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) f(x[k][j], i + k * kThreads, j);
    }
#pragma unroll 1
    for (; i < quads; i += kThreads) {
      float x[4];
      load(i, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f(x[j], i, j);
    }
  };

  // ---- the maximum; NaN counts as -infinity, +infinity as the type's largest number
  float top = -INFINITY;
  bool odd = false;
  sweep([&](float x, int, int) {
    top = fmaxf(top, x);
    odd |= !(x <= kMost);
  });
  clean = !__syncthreads_or(odd);
  if (HELD && !clean) {
#pragma unroll 1
    for (int i = tid; i < 4 * quads; i += kThreads) {
      if (F32) {
        float& x = reinterpret_cast<float*>(slice)[i];
        if (!(x <= kMost)) x = x != x ? -INFINITY : kMost;
      } else {
        uint16_t& w = reinterpret_cast<uint16_t*>(slice)[i];
        const float x = bf16_bits_to_f32(w);
        if (!(x <= kMost)) w = x != x ? (uint16_t)0xFF80u : (uint16_t)0x7F7Fu;
      }
    }
    __syncthreads();
  }
  top = fminf(top, largest);
  top = cta_all(top, Max(), partf);
  if (HELD) cluster_wait();
  if (tid < cluster) {
    tell32(&row.max[rank], tid, __float_as_uint(top));
    tell32(&row.landed[rank], tid, landed);
  }
  all_sync();
  for (int c = 0; c < cluster; ++c) top = fmaxf(top, row.max[c]), landed &= row.landed[c] != 0;

  // the whole cluster's sum; `which` alternates between calls, so that one's numbers are read before they are written again
  int turn = 0;
  auto cluster_sum = [&](u64 v) {
    v = cta_all(v, Add(), part64);
    turn ^= 1;
    if (tid < cluster) tell64(&row.sum[turn][rank], tid, v);
    all_sync();
    v = 0;
    for (int c = 0; c < cluster; ++c) v += row.sum[turn][c];
    return v;
  };

  int token = -1;
  float prob = 0.f;
  if (top == -INFINITY || !landed) {
    // nothing to draw
  } else if (greedy) {
    int at = 0x7FFFFFFF;
    sweep_slow([&](float x, int i, int j) {
      if (x == top) at = min(at, index_of(i, j));
    });
    at = cta_all(at, Min(), part32);
    if (tid < cluster) tell32(&row.lowest[rank], tid, (uint32_t)at);
    all_sync();
    for (int c = 0; c < cluster; ++c) at = min(at, row.lowest[c]);
    token = at;
    prob = 1.f;
  } else {
    Scale s;
    s.max = top;
    s.sj = sj;
    s.ch = step_of[0], s.cl = step_of[1];
    s.per = 0.69314718f / (float)(64 << s.sj);
    s.inv = -1.f / (float)(64 << s.sj);
    s.end = (float)(45 * 64 << s.sj);
    // x passes min_p from here on
    if (has_m) {
      if (tid == 0) least_at = __double2float_ru((double)top + least_of);
      __syncthreads();
    }
    const float least = has_m ? least_at : -INFINITY, p_share = fmaxf(p_raw, 0.f);
    auto share = [](float f, u64 z) { return times(f, z, true); };      // of a sum, for C >= share
    auto past = [](float f, u64 z) { return times(f, z, false) + 1; };  // for C > f z

    u64 Z = 0, drawn_of = 0;  // all weights; the kept ones
    int finite = 0;           // tokens above -infinity
    bool few = k > 0 && k <= kFewK;  // the bins only count, and are of the logits' scale
    bool done = false;
    float c_bin = 0.f;
    float drawn = 0.f;  // the token's logit

    // ---- the bins and what lies before each of this CTA's own
    auto histogram = [&]() {
      c_bin = few ? kFewScale : s.ch;
#pragma unroll 1
      for (int i = tid; i < kCopies * 2 * kBins / 4; i += kThreads) reinterpret_cast<int4*>(cnt)[i] = make_int4(0, 0, 0, 0);
      if (tid == 0) tail_of = 0;
      __syncthreads();
      int over = 0;
      uint32_t below = 0;
      u64 tail = 0;
      if (few) {
        sweep([&](float x, int, int) {
          const int b = bin_of(top - x, c_bin);
          if (b < kOver)
            atomicAdd(my_cnt + b, 1);
          else
            over += x > -INFINITY;
        });
      } else {
        sweep([&](float x, int, int) {
          const float d = top - x, th = d * s.ch, bm = fminf(th, (float)kOver) + kMagic;
          const int b = __float_as_int(bm) & 0xFFF;
          if (b < kOver) {
            int shift;
            const float middle = bm - kMagic, factor = steps_of(s, middle_f32(s, middle), shift);
            atomicAdd(my_cnt + b, 1);
            atomicAdd(my_dev + b, steps_below(s, x, d, middle, factor));
          } else {
            over += x > -INFINITY;
            below += weight_below(s, th);
          }
        });
        tail = below;
        if (s.sj > 0 && over) {  // (apart: in the sweep, this code slowed it down where it does not run)
          tail = 0;
          sweep_slow([&](float x, int, int) {
            if ((top - x) * s.ch > (float)kOver - 0.5f) tail += weight_of(s, pow, x);
          });
        }
      }
      over = warp_all(over, Add());
      const u64 tail_part = warp_all(tail, Add());
      if (lane == 0 && over) {
        atomicAdd(cnt + kOver, over);
        atomicAdd(&tail_of, tail_part);
      }
      all_sync();  // all counts are there
      // this CTA's bins, over the cluster: four or fewer consecutive ones a thread
      const int per = (own_bins + kThreads - 1) / kThreads, b0 = tid * per;
      int mine_n = 0;
      u64 mine_m = 0;
#pragma unroll 1
      for (int i = b0; i < min(b0 + per, own_bins); ++i) {
        const int b = rank * own_bins + i;
        int count = 0;
        long long deviate = 0;
        if (!HELD) count = cnt[2 * kBins + b], deviate = dev[2 * kBins + b];
#pragma unroll
        for (int r = 0; r < (HELD ? kMaxCluster : 1); ++r) {
          if (r < cluster) {
            count += (int)ask32(cnt + b, r);
            if (!few) deviate += (int)ask32(dev + b, r);
          }
        }
        before_n[i] = mine_n;
        before_m[i] = mine_m;
        if (b == kOver) {
          over = count;
          break;
        }
        mine_n += count;
        if (!few && count) {
          int shift;
          const float middle = middle_f32(s, (float)b);
          steps_of(s, middle, shift);
          mine_m += (u64)count * middle_of(pow, middle, b, s.sj) - (u64)(deviate * (1ll << shift));
        }
      }
      // exclusive sums over the threads
      if (b0 + per >= own_bins && b0 < own_bins && rank == cluster - 1)
        for (int r = 0; r < cluster; ++r) tell32(&row.over, r, (uint32_t)over);
      int inc_n = mine_n;
      u64 inc_m = mine_m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc_n, o);
        const u64 y = __shfl_up_sync(0xffffffffu, inc_m, o);
        if (lane >= o) inc_n += x, inc_m += y;
      }
      __syncthreads();
      if (lane == 31) part32[warp] = inc_n, part64[warp] = inc_m;
      __syncthreads();
      int base_n = inc_n - mine_n, total_n = 0;
      u64 base_m = inc_m - mine_m, total_m = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base_n += part32[w], base_m += part64[w];
        total_n += part32[w], total_m += part64[w];
      }
      if (tid < cluster) {
        tell32(&row.count[rank], tid, (uint32_t)total_n);
        tell64(&row.mass[rank], tid, total_m);
        tell64(&row.tail[rank], tid, tail_of);
      }
      all_sync();  // (and all have read the counts: a list may take their place)
      finite = row.over, Z = 0;
      for (int r = 0; r < cluster; ++r) {
        if (r < rank) base_n += row.count[r], base_m += row.mass[r];
        finite += row.count[r];
        Z += row.mass[r] + row.tail[r];
      }
#pragma unroll 1
      for (int i = b0; i < min(b0 + per, own_bins); ++i) before_n[i] += base_n, before_m[i] += base_m;
      __syncthreads();
    };
    // tokens, weight before the overflow bin
    auto inner_n = [&]() {
      int x = 0;
      for (int r = 0; r < cluster; ++r) x += row.count[r];
      return x;
    };
    auto inner_m = [&]() {
      u64 x = 0;
      for (int r = 0; r < cluster; ++r) x += row.mass[r];
      return x;
    };
    auto end_n = [&](int i) {  // after this CTA's bin i
      int x = 0;
      if (i + 1 < own_bins) return before_n[i + 1];
      for (int r = 0; r <= rank; ++r) x += row.count[r];
      return x;
    };
    auto end_m = [&](int i) {
      u64 x = 0;
      if (i + 1 < own_bins) return before_m[i + 1];
      for (int r = 0; r <= rank; ++r) x += row.mass[r];
      return x;
    };
    int search_turn = 0;
    // what this CTA knows of its bin i to the whole cluster
    auto tell = [&](int i) {
#pragma unroll 1
      for (int r = 0; r < cluster; ++r) {
        Found* f = &row.found[search_turn];
        tell32(&f->bin, r, (uint32_t)(rank * own_bins + i));
        tell32(&f->n, r, (uint32_t)before_n[i]);
        tell32(&f->count, r, (uint32_t)(end_n(i) - before_n[i]));
        tell64(&f->mass, r, before_m[i]);
        tell64(&f->after, r, end_m(i));
      }
    };
    // the bin in which the count (which 0) or the sum (1) reaches `want`; kOver where none of the inner ones does
    auto find = [&](int which, u64 want) {
      search_turn ^= 1;
#pragma unroll 1
      for (int i = tid; i < own_bins; i += kThreads) {
        const u64 lo = which ? before_m[i] : (u64)before_n[i], hi = which ? end_m(i) : (u64)end_n(i);
        if (lo < want && want <= hi) tell(i);
      }
      all_sync();
      Found f = row.found[search_turn];
      if (want > (which ? inner_m() : (u64)inner_n())) f.bin = kOver, f.n = inner_n(), f.count = finite - f.n, f.mass = inner_m(),
        f.after = Z;
      return f;
    };
    auto of_bin = [&](int b) {
      search_turn ^= 1;
      if (b / own_bins == rank && tid == b % own_bins % kThreads) tell(b % own_bins);
      all_sync();
      return row.found[search_turn];
    };
    // The first `count` of kList keys, place 32 (kPlaces warp + p) + lane of them in v[p], no two alike, into sorted[] in
    // descending order: parted by up to 32 of them (a key's part: how many of those are above it), then each one's place is
    // its part's beginning and the number of larger ones there. Whatever the parts are, the order is the same. (253 keys
    // 3.0, 622 6.9 thousand cycles; by a bitonic network 5.3 and 10.3, and unrolled no less: code that runs once is slow.)
    auto sort = [&](const u64 (&v)[kPlaces], int count) {
      const float scale = fminf(32.f / (float)count, 1.f);
      const int at = 32 * kPlaces * warp + lane;
#pragma unroll
      for (int p = 0; p < kPlaces; ++p) {
        const int i = at + 32 * p, k = (int)((float)i * scale);
        if (i < count && (i == 0 || (int)((float)(i - 1) * scale) < k)) splitter[k] = v[p];
      }
      if (tid >= count && tid < 32) splitter[tid] = 0ull;
      if (tid < 33) part_size[tid] = 0;
      __syncthreads();
      int part[kPlaces], nth[kPlaces];
#pragma unroll
      for (int p = 0; p < kPlaces; ++p) part[p] = 0;
      if (at < count) {
#pragma unroll 4
        for (int k = 0; k < 32; k += 2) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(splitter + k);
#pragma unroll
          for (int p = 0; p < kPlaces; ++p) part[p] += (x.x > v[p]) + (x.y > v[p]);
        }
      }
#pragma unroll
      for (int p = 0; p < kPlaces; ++p)
        if (at + 32 * p < count) nth[p] = atomicAdd(part_size + part[p], 1);
      __syncthreads();
      int upto = part_size[lane];
      const int own = upto;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      if (warp == 0) {
        part_begin[lane] = upto - own;
        if (lane == 31) part_begin[32] = upto, part_begin[33] = count;
      }
#pragma unroll
      for (int p = 0; p < kPlaces; ++p) {
        const int before = __shfl_sync(0xffffffffu, upto, max(part[p] - 1, 0));
        if (at + 32 * p < count) {
          const int to = nth[p] + (part[p] ? before : 0);
          list[to] = v[p];
          part_of[to] = (uint8_t)part[p];
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < count; i += kThreads) {
        const u64 key = list[i];
        const int from = part_begin[part_of[i]], to = part_begin[part_of[i] + 1];
        int place = from;
#pragma unroll 1
        for (int q = from; q < to; q += 4) {  // (a list's end is followed by sorted[])
          u64 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = list[q + k];
#pragma unroll
          for (int k = 0; k < 4; ++k) place += q + k < to && x[k] > key;
        }
        sorted[place] = key;
      }
      __syncthreads();
    };
    // the CTAs' lists, of which row.listed tells, sorted in CTA 0; their number
    auto collect = [&]() {
      int ends[kMaxCluster], count = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        if (r < cluster) count += row.listed[r];
        ends[r] = count;
      }
      count = min(count, kList);
      u64 v[kPlaces];
#pragma unroll
      for (int p = 0; p < kPlaces; ++p) {  // all on the way at once
        const int i = 32 * (kPlaces * warp + p) + lane;
        int r = 0, begin = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster - 1; ++q)
          if (i >= ends[q]) r = q + 1, begin = ends[q];
        v[p] = i < count ? ask64(list + i - begin, r) : 0ull;
      }
      sort(v, count);
      return count;
    };
    auto put_in_list = [&](float x, int i, int j) {
      const int at = atomicAdd(&taken, 1);
      if (at < kList) list[at] = (u64)key_of(x) << 32 | (uint32_t)~index_of(i, j);
    };
    // The tokens of bins lo .. hi and of bin `too`, no more than kList of them, sorted in CTA 0: keys in descending order
    // with the complement of the index below.
    auto gather = [&](int lo, int hi, int too) {
      if (tid == 0) taken = 0;
      __syncthreads();
      sweep([&](float x, int i, int j) {
        const int b = bin_of(top - x, c_bin);
        if (((b >= lo && b <= hi) || b == too) && x > -INFINITY) put_in_list(x, i, j);
      });
      __syncthreads();
      if (tid == 0) tell32(&row.listed[rank], 0, (uint32_t)min(taken, kList));
      all_sync();
      return rank == 0 ? collect() : 0;
    };
    // In CTA 0, of a sorted list: the sums of the weights up to each of the thread's places, kPlaces tid and on
    struct Sums {
      u64 at[kPlaces];
    };
    auto prefix = [&](int count) {
      Sums sum;
      u64 inc = 0;
#pragma unroll
      for (int j = 0; j < kPlaces; ++j) {
        const int i = kPlaces * tid + j;
        inc += i < count ? weight_of(s, pow, value_of((uint32_t)(sorted[i] >> 32))) : 0ull;
        sum.at[j] = inc;
      }
      const u64 own = inc;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) part64[warp] = inc;
      __syncthreads();
      inc -= own;
#pragma unroll
      for (int v = 0; v < kWarps; ++v)
        if (v < warp) inc += part64[v];
#pragma unroll
      for (int j = 0; j < kPlaces; ++j) sum.at[j] += inc;
      return sum;
    };
    // smallest place from .. count - 1 of a list at which base + its sum reaches `want` (count if none does): for CTA 0's
    // threads
    auto reach_from = [&](const Sums& sum, int from, int count, u64 base, u64 want) {
      int at = count;
#pragma unroll
      for (int j = kPlaces - 1; j >= 0; --j)
        if (kPlaces * tid + j >= from && kPlaces * tid + j < count && base + sum.at[j] >= want) at = kPlaces * tid + j;
      return cta_all(at, Min(), part32);
    };
    auto reach = [&](const Sums& sum, int count, u64 base, u64 want) { return reach_from(sum, 0, count, base, want); };
    auto sum_at = [&](const Sums& sum, int i) {  // the sum at place i, for all threads of CTA 0
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPlaces; ++j)
        if (kPlaces * tid + j == i) row.result[0] = sum.at[j];
      __syncthreads();
      return row.result[0];
    };
    // In CTA 0, the token of a list that begins with all that is kept (of the k first where `by_k`). Where Z is known but
    // to `slack`, false unless top-p's end lies in the list and is the same for all that Z may be (or min_p's comes first).
    auto draw = [&](int count, bool by_k, u64 slack) {
      const Sums sum = prefix(count);
      int keep = by_k ? min(k, count) : count, pass = count;
      if (has_m) {
        pass = 0;
#pragma unroll
        for (int j = 0; j < kPlaces; ++j)
          pass += kPlaces * tid + j < count && value_of((uint32_t)(sorted[kPlaces * tid + j] >> 32)) >= least;
        pass = cta_all(pass, Add(), part32);
      }
      if (has_p) {
        const u64 z = by_k ? sum_at(sum, keep - 1) : Z - slack;
        const int at = reach(sum, keep, 0, max(1ull, share(p_share, z)));
        if (slack && (pass == count || at < pass) && (at == count || sum_at(sum, at) < share(p_share, Z + slack))) return false;
        keep = min(keep, at + 1);
      }
      keep = min(keep, pass);
      keep = max(keep, 1);
      drawn_of = sum_at(sum, keep - 1);
      const int at = min(reach(sum, keep, 0, past(u, drawn_of)), keep - 1);
      token = (int)~(uint32_t)sorted[at];
      drawn = value_of((uint32_t)(sorted[at] >> 32));
      return true;
    };

    // ---- where a bin holds more than a list does, or the target lies below the bins: by halving the numbers that the
    // order's keys, then the indexes of equal ones, may be (slow, for rows of many equal logits, or very flat ones)
    auto mass_from = [&](uint32_t key) {
      u64 w = 0;
      sweep_slow([&](float x, int, int) {
        if (key_of(x) >= key) w += weight_of(s, pow, x);
      });
      return cluster_sum(w);
    };
    auto count_from = [&](uint32_t key) {
      u64 w = 0;
      sweep_slow([&](float x, int, int) { w += key_of(x) >= key && x > -INFINITY; });
      return cluster_sum(w);
    };
    // the sum at the place where the count (which 0) or the sum reaches `want`, and that place's key and number among its
    // equals
    struct Place {
      u64 sum;
      uint32_t key;
      u64 nth;
    };
    auto search = [&](int which, u64 want) {
      uint32_t lo = key_of(-kMost), hi = key_of(top);  // the largest key from which on it is reached lies here
#pragma unroll 1
      while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        if ((which ? mass_from(mid) : count_from(mid)) >= want)
          lo = mid;
        else
          hi = mid - 1;
      }
      Place r;
      r.key = lo;
      const u64 w = weight_of(s, pow, value_of(lo)), m_above = lo == 0xFFFFFFFFu ? 0 : mass_from(lo + 1),
                n_above = lo == 0xFFFFFFFFu ? 0 : count_from(lo + 1), equal = count_from(lo) - n_above;
      r.nth = which ? (w ? (want - min(want, m_above) + w - 1) / w : 1ull) : want - min(want, n_above);
      r.nth = max(1ull, min(r.nth, equal));
      r.sum = m_above + r.nth * w;
      return r;
    };
    auto index_of_nth = [&](uint32_t key, u64 nth) {
      int lo = 0, hi = a.V - 1;
#pragma unroll 1
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        u64 w = 0;
        sweep_slow([&](float x, int i, int j) { w += key_of(x) == key && index_of(i, j) <= mid; });
        if (cluster_sum(w) >= nth)
          hi = mid;
        else
          lo = mid + 1;
      }
      return lo;
    };

    // ---- Short of counting all tokens: a bound below which a few hundred lie above is guessed from a sample, and what
    // lies above it gathered, with about the sum of all weights where top-p needs that. If what is kept proves to reach
    // further, if it would end elsewhere with a little more or less of that sum, or if the bound is far off, the bins below
    // decide.
    const bool every = a.V <= kList;  // a list holds the whole row
    if (every || (k ? k <= kList / 2 : has_p || has_m)) {
      bool hopeless = false;
      float bound = -kMost;
      if (!every && !k && !has_p) {
        bound = fmaxf(least, -kMost);
      } else if (!every) {
        // The r-th largest of the warps' largest sampled logits: of 16 warps' samples together about the
        // 16 (1 / 16 + .. + 1 / (17 - r))-th largest (and so with 32). A thread samples one quad.
        float best = -INFINITY, x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const int i = quads > kThreads ? (int)((long long)tid * quads / kThreads) : tid;
        if (i < quads) {
          load(i, x);
          best = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        }
        best = warp_all(best, Max());
        __syncthreads();
        if (lane == 0) partf[warp] = best;
        __syncthreads();
        const float want = (float)(k ? max(160, 3 * k) : 300) / (float)cluster * (float)kThreads / (float)max(quads, kThreads);
        int r = 0;
        for (float at = 0.f; r < kWarps && at < want; ++r) at += (float)kWarps / (float)(kWarps - r);
        r = max(r, 1);
        const float mine = partf[lane & (kWarps - 1)];
        int above = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) above += partf[w] > mine || (partf[w] == mine && w < (lane & (kWarps - 1)));
        const unsigned it = __ballot_sync(0xffffffffu, above == r - 1);
        bound = __shfl_sync(0xffffffffu, mine, __ffs(it) - 1);
        // With top-p alone, the weights below the bound as the sample has them: where they outweigh some 250 of the largest
        // (1 - p) / p times what lies above is too little.
        float below = 0.f;
        if (has_p && !k) {
#pragma unroll
          for (int j = 0; j < 4; ++j) below += x[j] < bound ? ex2((x[j] - top) * s.ch / (float)(64 << s.sj)) : 0.f;
          below = cta_all(below, Add(), part_below) * (float)max(quads, kThreads) / (float)kThreads;
        }
        // the middle one of the CTAs'
        if (tid < cluster) {
          tell32(&row.bound[rank], tid, __float_as_uint(bound));
          tell32(&row.below[rank], tid, __float_as_uint(below));
        }
        all_sync();
        const float theirs = row.bound[lane & (cluster - 1)];
        int more = 0;
        for (int o = 0; o < cluster; ++o) {
          const float x = __shfl_sync(0xffffffffu, theirs, o);
          more += x > theirs || (x == theirs && o < (lane & (cluster - 1)));
        }
        const float middle_one = __shfl_sync(0xffffffffu, theirs, __ffs(__ballot_sync(0xffffffffu, more == cluster / 2)) - 1);
        bound = fmaxf(middle_one, -kMost);
        below = 0.f;
        for (int o = 0; o < cluster; ++o) below += row.below[o];
        hopeless = below * p_share > 250.f * (1.f - p_share) && !has_m;
      }
      if (!hopeless) {
        if (tid == 0) taken = 0;
        __syncthreads();
        u64 mass = 0;
        float four = 0.f, above = 0.f;
        const float c1 = -s.ch / (float)(64 << s.sj), c2 = -s.cl / (float)(64 << s.sj);
        const bool need_z = has_p && !k && !every;
        sweep([&](float x, int i, int j) {
          if (x >= bound) put_in_list(x, i, j);
          if (need_z) {
            const float d = top - x, w = ex2(fmaxf(fmaf(d, c1, d * c2), -200.f));  // (of -infinity that sum is no number)
            // (By fours as whole numbers: whatever the row, Z is off by less than 2^-18 of itself. w's exponent is rounded twice
            // to 2^-24 of itself: a octaves below the maximum that is 2^-23.5 a of w, and what lies there weighs at most
            // 2^(18.6 - a), so of Z it is 2^-19.7 at most; ex2 adds 2^-22, three additions 2^-22.4, units cut off 2^-25.)
            four = j ? four + w : w;
            if (j == 3) mass += (u64)(four * 8796093022208.f);  // 2^43
            above += x >= bound ? w : 0.f;
          }
        });
        const u64 mine = need_z ? cta_all(mass, Add(), part64) : 0ull;
        const u64 listed = need_z ? cta_all((u64)(above * 8796093022208.f), Add(), part64) : 0ull;
        __syncthreads();
        if (tid < cluster) {
          tell32(&row.listed[rank], tid, (uint32_t)taken);
          tell64(&row.mass[rank], tid, mine);
          tell64(&row.tail[rank], tid, listed);
        }
        all_sync();
        int count = 0;
        u64 in_list = 0;
        for (int r = 0; r < cluster; ++r) count += row.listed[r], Z += row.mass[r], in_list += row.tail[r];
        // (a list that ends before top-p and min_p do is not worth sorting)
        const bool far = !need_z || (has_m && least >= bound) || in_list + (Z >> 10) >= share(p_share, Z);
        if (far && count > 0 && count <= kList && (count >= k || every)) {
          bool ok = true;
          if (rank == 0) {
            count = collect();
            if (every) {  // (all weights, and k as if there were no more than that)
              const Sums sum = prefix(count);
              Z = sum_at(sum, count - 1);
            }
            ok = draw(count, k > 0, need_z ? Z >> 18 : 0ull);
          }
          if (need_z) {
            if (tid < cluster && rank == 0) tell32(&row.done, tid, ok);
            all_sync();
            ok = row.done != 0;
          }
          done = ok;
        }
      }
      if (!done) Z = 0;
    }

    // ---- small cuts: all that may be kept in one list
    Found kth = {}, pth = {};
    bool has_k = false;
    if (!done) {
    histogram();
    if (k && k < finite) kth = find(0, (u64)k);
    if (few && (k >= finite || kth.bin == kOver || kth.n + kth.count > kList)) {
      // the k-th does not lie in a list's reach: bins of weights
      few = false;
      histogram();
      if (k && k < finite) kth = find(0, (u64)k);
    }
    has_k = k && k < finite;
    int last = kOver, upto = kList + 1;  // a bin that holds the end of what is kept, and the tokens up to its end
    if (has_k) {
      last = kth.bin, upto = kth.n + kth.count;
    } else if (has_p) {
      pth = find(1, max(1ull, share(p_share, Z)));
      last = pth.bin, upto = pth.n + pth.count;
    }
    if (has_m && !(has_k && has_p)) {  // (top-p after top-k needs the k first)
      const int b = bin_of(top - fmaxf(least, -kMost), c_bin) + 1;
      if (b < kOver && b < last) {
        const Found f = of_bin(b);
        last = b, upto = f.n + f.count;
      }
    }
    if (last != kOver && upto <= kList) {
      const int count = gather(0, last, 0);
      if (rank == 0) draw(count, has_k, 0);
      done = true;
    }
    }
    if (!done) {
      // ---- large cuts, or none: each one's end lies in one bin
      drawn_of = Z;
      auto end_of = [&](int which, const Found& f, u64 want) {  // the sum at the place where it reaches `want`
        if (f.bin == kOver || f.count > kList) return search(which, want).sum;
        const int count = gather(f.bin, f.bin, f.bin);
        if (rank == 0) {
          const Sums sum = prefix(count);
          int at = which ? reach(sum, count, f.mass, want) : (int)(want - f.n) - 1;
          at = min(max(at, 0), count - 1);
          const u64 z = f.mass + sum_at(sum, at);
          if (tid < cluster) tell64(&row.result[1], tid, z);
        }
        all_sync();
        return row.result[1];
      };
      if (has_k) drawn_of = end_of(0, kth, (u64)k);
      if (has_p) {
        const u64 want = max(1ull, share(p_share, drawn_of));
        const Found f = pth.mass < want && want <= pth.after ? pth : find(1, want);
        // Wherever in its bin top-p ends, the draw ends in one bin or a few: they are gathered at once (a sweep and a sort
        // less).
        const bool at_once = !has_m && f.bin != kOver;
        const u64 most = past(u, min(drawn_of, f.after));
        const Found d = at_once ? find(1, past(u, min(drawn_of, want))) : f,
                    e = at_once && most > d.after ? find(1, most) : d;
        const int ahead = e.bin < f.bin ? e.n + e.count - d.n : f.n - d.n;  // tokens listed before those of top-p's bin
        if (at_once && d.bin <= f.bin && ahead + f.count <= kList) {
          const int count = gather(d.bin, min(e.bin, f.bin), f.bin);
          if (rank == 0) {
            const Sums sum = prefix(count);
            const u64 base = f.mass - (ahead ? sum_at(sum, ahead - 1) : 0ull);
            const int end = min(reach_from(sum, ahead, count, base, want), count - 1);
            drawn_of = min(drawn_of, base + sum_at(sum, end));
            const int upto = e.bin < f.bin ? ahead : count, at = min(reach(sum, upto, d.mass, past(u, drawn_of)), upto - 1);
            token = (int)~(uint32_t)sorted[at];
            drawn = value_of((uint32_t)(sorted[at] >> 32));
          }
          done = true;
        } else {
          drawn_of = min(drawn_of, end_of(1, f, want));
        }
      }
      if (!done) {
        if (has_m) drawn_of = min(drawn_of, mass_from(key_of(fmaxf(least, -kMost))));
        const u64 want = past(u, drawn_of);
        const Found f = find(1, want);
        if (f.bin == kOver || f.count > kList) {
          const Place at = search(1, want);
          token = index_of_nth(at.key, at.nth);
          drawn = value_of(at.key);
        } else {
          const int count = gather(f.bin, f.bin, f.bin);
          if (rank == 0) {
            const Sums sum = prefix(count);
            const int at = min(reach(sum, count, f.mass, want), count - 1);
            token = (int)~(uint32_t)sorted[at];
            drawn = value_of((uint32_t)(sorted[at] >> 32));
          }
        }
      }
    }
    if (rank == 0 && tid == 0)
      prob = share_of(s, pow, drawn, drawn_of);
  }
  if (rank == 0 && tid == 0) {
    a.tokens[m] = token;
    if (a.probs) a.probs[m] = prob;
  }
  all_sync();  // no CTA leaves while another reads its memory
  if (!landed) mbar_wait_n(&bar, 0, nullptr, 0, 1u << 16);  // nor before its copies have landed (a bounded wait)
}

// Where a CTA per row pays: the clusters' rows follow one another through the SMs, 2 SMs / cluster at a time and some 20 us
// each, mostly waiting for their own barriers; a CTA per row takes 8 us and 0.43 ns a logit, but the GPU holds two an SM.
// Clusters of 8 and CTAs of 512 threads, plain softmax, fp32: 76 rows of 20001 logits 46.5 and 20.5 us, of 50021 50.8 and
// 32.9, of 151936 65.5 and 72.1; 128 rows of 151936 98.7 and 72.6, 152 rows 113 and 73, 512 rows 354 and 252. (The counts
// of one of the two copies of the bins stay below 2^31 / 22780 = 94270, that a bin's deviations fit 32 bits.)
bool row_per_cta(long long M, int V, int cluster) {
  return V <= 180000 && 152 * M * cluster > (long long)device_sm_count() * (120 + V / 154);
}

size_t sample_smem(bool f32, int V, int cluster) {
  return 2 * kBins * 4 + kBins / cluster * 12 + 16 * ((size_t)(V / (f32 ? 4 : 8) + cluster - 1) / cluster + 3);
}

template <bool F32>
cudaError_t launch(const SampleArgs& a, cudaStream_t stream, bool pdl) {
  const int sms = device_sm_count(), most = a.V <= 8192 ? 1 : a.V <= 16384 ? 2 : a.V <= 32768 ? 4 : 8;
  // the largest cluster with which all rows are held at once, a CTA an SM, if there is one (plain softmax, 76 rows of 50021
  // logits: clusters of 8, 4, 2, a CTA per row that reads it from L2: 51, 35, 22, 33 us; with 1024 threads a CTA 30)
  int cluster = most;
  auto ctas = [&](int c) {
    const size_t bytes = sample_smem(F32, a.V, c) + 4 * 1024;
    return bytes <= (size_t)device_max_smem_optin() && a.V / c <= 94000 ? sms : 0;
  };
  while (cluster > 1 && (long long)a.M * cluster > ctas(cluster)) cluster /= 2;
  bool held = (long long)a.M * cluster <= ctas(cluster);
  if (!held) cluster = most, held = cluster == 1 || !row_per_cta(a.M, a.V, cluster);
  // Two CTAs an SM; where their rows together would not stay in L2, one of 1024 threads (512 rows of 50021 fp32 logits:
  // two of 512 threads an SM 90.6 us, one of 1024 118; 76 rows of 151936 72.1 and 59.6, 152 rows 72.9 and 63.5, 512 rows
  // 252 and 253, with top-k 50 152 rows 76.8 and 33.7).
  const bool much = 2ll * sms * a.V * (F32 ? 4 : 2) > 96ll << 20;
  const int threads = !held && much ? 1024 : 512;
  auto k = held ? sample_kernel<F32, true, 512> : much ? sample_kernel<F32, false, 1024> : sample_kernel<F32, false, 512>;
  cudaError_t e = allow_max_smem(k);
  if (e != cudaSuccess) return e;
  if (!held) return launch_kernel(k, dim3(a.M), dim3(threads), 4 * kBins * 4 + kBins * 12, stream, pdl, a, 1);
  const size_t smem = sample_smem(F32, a.V, cluster);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.M * cluster);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a, cluster);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t stream, bool pdl) {
  return a.f32 ? launch<true>(a, stream, pdl) : launch<false>(a, stream, pdl);
}

}  // namespace qg
