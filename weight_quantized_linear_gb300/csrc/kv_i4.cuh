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

// Eight codes of a row as fp16 values code * s + lo, each rounded once (what kv_read_i4 gives), in the order of their
// nibbles: channels (0, 4), (1, 5), (2, 6), (3, 7).  A code in the low bits of an fp16 number between 1024 and 2048 is that
// code or 16 times it above 1024, so one masked merge and one exact operation make it a number.
__device__ __forceinline__ void kv_values8(uint32_t w, uint32_t s2, uint32_t lo2, uint32_t (&v)[4]) {
  const uint32_t w8 = w >> 8;
  v[0] = hfma2_u32(hadd2_u32(and_or(w, 0x000f000fu, 0x64006400u), 0xE400E400u), s2, lo2);
  v[1] = hfma2_u32(hfma2_u32(and_or(w, 0x00f000f0u, 0x64006400u), 0x2C002C00u, 0xD400D400u), s2, lo2);
  v[2] = hfma2_u32(hadd2_u32(and_or(w8, 0x000f000fu, 0x64006400u), 0xE400E400u), s2, lo2);
  v[3] = hfma2_u32(hfma2_u32(and_or(w8, 0x00f000f0u, 0x64006400u), 0x2C002C00u, 0xD400D400u), s2, lo2);
}
// For mma.sync: the token (of 16) that row r of an 8 x 8 block of weights stands for; K's rows, V's reduction index and the
// params all use it.  Chosen so that the shared-memory loads of K and V hit every bank once.
template <int D>
__device__ __forceinline__ int token_of(int r) {
  const int c = r >> 1, e = r & 1;
  return 2 * c + (e ^ (D == 128 ? (c & 1) : (c >> 1)));
}
// A finite row may hold values that round to infinity (its s may have been rounded up); attention over fp16 values takes
// the largest finite number for them.  What of a row's parameters says that.
__device__ __forceinline__ bool kv_finite(uint32_t par) { return ((par & 0x7c007c00u) + 0x04000400u & 0x80008000u) == 0; }
__device__ __forceinline__ bool kv_overflows(uint32_t par) {  // for finite parameters
  const float s = __half2float(__ushort_as_half((unsigned short)par)), lo = __half2float(__ushort_as_half((unsigned short)(par >> 16)));
  return fabsf(fmaf(15.f, s, lo)) >= 65520.f;
}
__device__ __forceinline__ uint32_t kv_clamp2(uint32_t v) {
  const __half2 x = *reinterpret_cast<const __half2*>(&v), m = __half2half2(__ushort_as_half(0x7bff));
  const __half2 y = __hmax2_nan(__hmin2_nan(x, m), __hneg2(m));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// A sequence of packed chunks: rows start .. start + rows - 1 of q are the last `rows` of its `len` tokens; row r sees the
// tokens up to first + r, first = len - rows.  Out of range: no rows, or the length that the table holds.
struct KvChunk {
  int start, rows, len, first;
};
__device__ __forceinline__ KvChunk kv_chunk(const int* cu, const int* kv_lens, int b, int T, int cap, unsigned* err) {
  const int s = cu[b], e = cu[b + 1];
  int len = max(kv_lens[b], 0);
  if (len > cap) {
    report_error(err, kErrBadIndex);
    len = cap;
  }
  if (s < 0 || e < s || e > T) {
    report_error(err, kErrBadIndex);
    return {0, 0, len, len};
  }
  return {s, e - s, len, len - (e - s)};
}

// Copy of `bytes` (a multiple of 16) from global to shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

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
