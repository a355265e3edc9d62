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

#include "attn_kv8_mma.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

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
  return format == QG_KV_I8 ? launch_by_shape<QG_KV_I8, false>(a, stream, pdl) : launch_by_shape<QG_KV_E4M3, false>(a, stream, pdl);
}

}  // namespace qg
