// How attn_kv8_prefix.cu cuts the prefixes of a batch, and where its pieces lie;
// attn_kv8_shared.cu joins them.
#pragma once

#include "attn_kv8.cuh"

namespace qg {
namespace {

constexpr int kPrefixRows = 256;  // query rows of an item
constexpr int kPrefixTok = 128;   // tokens of a step
using PrefixCut = AttnCut<kPrefixTok, 4, 1>;

// a piece: fp32 outputs [256][D], then (maximum, sum) [256]
__host__ __device__ constexpr size_t prefix_piece_bytes(int D) { return (size_t)kPrefixRows * (D * 4 + 8); }
__device__ __forceinline__ uint8_t* prefix_piece(void* pieces, int cta, int second, int D) {
  return static_cast<uint8_t*>(pieces) + (size_t)(2 * cta + second) * prefix_piece_bytes(D);
}

}  // namespace
}  // namespace qg
