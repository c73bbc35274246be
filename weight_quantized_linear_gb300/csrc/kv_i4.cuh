// kv_i4.cuh -- layout of the paged 4-bit KV cache, shared by its codec and the attention over it.
//
// The cache is [pages, heads, page_size / 16] blocks of 16 tokens of one K/V head, 16 (D + 8) bytes each:
//   K codes [16, D / 2]   channel 2i in the low half of byte i, channel 2i + 1 in the high half
//   V codes [16, D / 2]
//   K params [16] {fp16 s, fp16 lo},  V params [16] {fp16 s, fp16 lo}
// and a value is code * s + lo.  Everything that attention reads of 16 tokens is one contiguous run, so a
// run of blocks inside a page arrives by a single bulk copy, whatever the page size; 16 (D + 8) is a
// multiple of 128 for D = 64 and D = 128.
#pragma once

#include "common.cuh"

namespace wql {

constexpr int kKvBlock = 16;  // tokens per block

template <int D>
struct KvI4 {
  static constexpr int kRow = D / 2;                    // bytes of one token's codes
  static constexpr int kV = kKvBlock * kRow;            // offset of the V codes
  static constexpr int kKp = 2 * kKvBlock * kRow;       // offset of the K params
  static constexpr int kVp = kKp + 4 * kKvBlock;        // offset of the V params
  static constexpr int kBytes = kKvBlock * (D + 8);     // a block
};

// Division by a number known at launch: n / d for 0 <= n < 2^31 (Granlund and Montgomery's multiplier with l = ceil(log2 d)).
struct FastDiv {
  uint32_t d, m, l;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {d, (uint32_t)((((1ull << l) - d) << 32) / d + 1), l};
}
__device__ __forceinline__ uint32_t quot(uint32_t n, const FastDiv& f) { return (__umulhi(n, f.m) + n) >> f.l; }

}  // namespace wql
