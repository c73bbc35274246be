// attn_chunks_i4.cu -- attention of packed chunks of new tokens over the paged 4-bit KV cache, with grouped heads.
//
// Sequence b's chunk is rows cu[b] .. cu[b + 1] - 1 of q, the last ones of its kv_lens[b] tokens, all of which are in the
// cache.  For row r of n and query head h:
//   out = sum_t softmax_t(scale q . k[t]) v[t],   lse = ln sum_t exp(scale q . k[t]),   t <= kv_len - n + r
// with k and v of K/V head h / (Hq / Hkv): code * s + lo, rounded to fp16, which is what the matrix product takes.
//
// This file has the kernel for chunks of many rows and the one that joins parts; sequences with up to 8 or 16 rows per K/V head
// (tokens times the G query heads of a group) go to attn_steps_i4.cu, where 128-row tiles would be nearly empty.
//
// A tile is 128 / G tokens of one K/V head, each with its G query heads: up to 128 rows, all of which read the same keys.
// A CTA works on two tiles of consecutive tokens at a time.  Per 128 keys, the tensor cores compute S = Q K^T into tensor
// memory, the tile's four softmax warps turn it into weights P (thread r owns row r, so neither maximum nor sum needs an
// exchange) as fp16, and the tensor cores add P V to the tile's accumulator.  With heads of 128 tensor memory is full, P is written
// over S and the two tiles take turns at the tensor cores, one's softmax beside the other's products; with heads of 64 P has
// columns of its own and the next S need not wait for it.  Where a sequence's last tokens fill one tile only, both halves of the
// CTA work on that tile, one on the even and one on the odd key tiles, and are joined in tensor memory.
//
// The weights are computed by the maximum as it was and kept in registers until their sum has said that none is too large for
// fp16; only then is a new maximum looked for and the accumulator rescaled.  Looking for it in every step cost the time of reading
// S twice (512 tokens behind 15872: 143 -> 135 us with three raw slots; mixed batch with heads of 64: 128 -> 126).
//
// K and V reach the tensor cores by way of eight warps that make fp16 numbers of the codes: bulk copies bring the blocks of
// 64 tokens as they are into a slot of the group that converts them, a thread takes one key's row there and writes it as a row of
// a swizzled operand tile.
// That is 3.5 instructions per pair of values, done once for the 256 rows of a pair of tiles.
//
// The key tiles of all items, one behind the other, are divided evenly over the CTAs, one per SM, whatever the lengths: a CTA finds
// its first item by closed forms for what is before an item, not by walking.  One of both tiles of rows counts as much as one where
// the halves share a tile, although two of those are worked on at once: the conversion is the same, and two take 1.6 to 1.7 times as
// long (counted as one, the CTAs that had them ended last, mixed batch 126 us for 102).  What a CTA computes of an item that it
// shares with others goes to the workspace as (O, m, l), and the joining kernel adds the parts in their order, so results do not
// depend on who did what.
//
// Bound by the tensor cores' and the softmax's chain: with heads of 128 a round of two tiles takes about 3900 cycles for 2048 of
// products: a tile's softmax 1300, its turn, and 1300 in which its two products hold the tensor cores, since Q K^T and P V read
// both fp16 operand tiles from shared memory while the converting warps write the next (without the conversion 111 us instead of
// 136).  With heads of 64 a round takes 3600 for 1024: both softmaxes at once, 1024 of it exponentials.
// Roundings: weights are fp16 because the second product takes them beside V, which the formula has in fp16 anyway.  Outputs are off
// by 2.5e-4 of their norm, of which 2.1e-4 is their own rounding.  What the rounding leaves as another operand would leave that
// alone, for another product as large as P V in a kernel that waits for its products.  The sum is taken of the weights before
// they are rounded, in fp32; exponential and logarithm to base 2 are the GPU's approximations (2^-22), below what fp32 scores are
// off.  Measured: log-sums within 4e-6.
// Measured on GB300 through the Python call, rows of 32 query heads:
//   512 tokens behind 15872, 8 K/V heads of 128     142 us    955 TFLOP/s, 50 % of the measured peak
//   4 x 2048 tokens over 2048 to 8190, 32 heads     580 us    950 TFLOP/s
//   24 requests up to 6000 tokens, three chunks of about 500 among single tokens, 8 K/V heads of 64     104 us
//   16 tokens behind 700, 32 heads, in a q of 19 rows     15 us, launches and latency
// The last of these is a case of the rule at the end of this file: in a q of just its 16 rows the kernel for a few rows takes it,
// 16.3 us for 14.8 in a graph.
// What did not pay: the conversion's loop unrolled twice or four times (142 and 150 us for 135, with three raw slots: the warps' code no
// longer stays in the instruction caches), no turns (163).
#include <atomic>
#include <climits>

#include "attn.cuh"
#include "attn_chunks.cuh"
#include "internal.h"

namespace wql {
namespace {

constexpr int kTile = 128, kHalf = 64;  // keys of a tile, and rows at most; keys of a step of the copies
// warps 0-3, 4-7: softmax of tiles 0, 1; 8: copies; 9, 10: products of tiles 0, 1; 11: next item; 12-19: K and V to fp16
constexpr int kThreads = 640;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kNextWarp = 11, kConvWarp = 12;
constexpr int kLead = 1;             // key tiles that stand for an item's own cost
constexpr float kTop = 7.0f;         // the largest weight after a rescale is 2^7
constexpr float kMost = 32768.f;     // and a step whose weights come to more than 2^15 asks for the next,
constexpr float kLarge = 1048576.f;  // from here on scores are rounded before the maximum is subtracted, as it was
constexpr float kNoMax = -3e38f;     // the maximum of keys whose scores are all minus infinity
// registers per thread: launched with 96; two warpgroups for the softmax, two convert, one does the rest
constexpr int kSoftmaxRegs = 136, kConvRegs = 72, kOtherRegs = 56;
static_assert(2 * kSoftmaxRegs + 2 * kConvRegs + kOtherRegs <= 5 * 96, "of what the block was launched with");

template <int D>
struct Cfg {
  static constexpr int kBox = kTile * 128;          // 128 rows of 64 fp16, 128-byte swizzle
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;  // a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 4 : 8;   // of K and V tiles
  static constexpr int kRawBytes = kHalf / kKvBlock * KvI4<D>::kBytes;  // blocks as they are, of half a tile of keys
  // One raw slot for each of the two groups that convert, or three.  With an odd number a group would see every other phase of a slot's
  // barrier only, and could take an old one for the next.
  static constexpr int kRaw = D == 128 ? 2 : 6;
  static_assert(kRaw % 2 == 0, "a raw slot is one group's");
  static_assert(kSlots % 2 == 0, "a slot has K or V, so that its warps meet every phase of its barriers");
  // D = 64 leaves room in tensor memory for P beside S, so that the next S is computed while this one's softmax runs
  static constexpr bool kBeside = D == 64;
  static constexpr int kColO = 2 * kTile, kColP = kBeside ? kColO + 2 * D : 0;  // tensor memory columns; S from 0
  static constexpr int kStrideP = kBeside ? kTile / 2 : kTile;                  // between the tiles' P
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffRaw = kOffRing + kSlots * kTileBytes;
  static constexpr int kSmem = kOffRaw + kRaw * kRawBytes + 1024;  // and alignment of the start
  static_assert(kSmem <= 223 * 1024, "shared memory, 4 KB of it static");
};

struct Args {
  const int *cu, *kv_lens;
  int B, T, Hq, Hkv, G, tokens;  // tokens of a tile
  const uint8_t* cache;
  int pages, bpp;  // bpp: blocks of a page
  FastDiv by_bpp;
  const int* table;
  int width, cap;
  float scale_log2;
  uint32_t negate;  // bit of the instruction descriptor that negates Q, for a negative scale
  __half* out;
  float* lse;
  ChunkParts parts;
  int few;  // sequences of up to so many rows are not taken here
  unsigned* err;
};

// Key tiles of an item and what is before it in its sequence.  Tokens [A p, A p + A) of a chunk of n are item p, A = 2 a.tokens;
// its last row sees first + A p + (its tokens) keys.
struct Shape {
  int first, n, A, items;
  __device__ __forceinline__ Shape(const Args& a, const KvChunk& c)
      : first(c.first), n(c.rows), A(2 * a.tokens), items(c.rows > a.few ? (c.rows - 1) / (2 * a.tokens) + 1 : 0) {}
  __device__ __forceinline__ int count(int p) const { return min(n - p * A, A); }
  __device__ __forceinline__ int tiles(int p) const { return max(first + p * A + count(p) - 1, 0) / kTile + 1; }  // of keys
  __device__ __forceinline__ bool twin(int p) const { return 2 * count(p) <= A; }
  // Key tiles (kLead more for each) of items 0 .. p - 1, all of them whole, p < items: the sum over i of max(1, ceil(x / 128)) with
  // x = first + A (i + 1).
  __device__ long long before(int p) const {
    if ((A & (A - 1)) == 0) {  // the usual numbers of heads, and no division
      const int a = __ffs(A) - 1;
      const long long one = min(max(((long long)kTile - first) >> a, 0LL), (long long)p);  // items with a single round
      const long long y = (long long)first + kTile - 1;
      long long sum = (long long)p * kLead + one;
      if (a >= 7)
        sum += (p - one) * (y >> 7) + ((((long long)p * (p + 1) - one * (one + 1)) / 2) << (a - 7));
      else
        sum += floors((y >> a) + p + 1, 7 - a) - floors((y >> a) + one + 1, 7 - a);
      return sum;
    }
    const long long one = min(max(floor_div((long long)kTile - first, A), 0LL), (long long)p);
    // the sum of floors of (x k + y) / m by Euclid's steps on (A, 128)
    long long sum = (long long)p * kLead + one, n_ = p - one, m = kTile, x = A, y = A * one + (long long)first + A + kTile - 1;
    while (n_ > 0) {
      if (x >= m) sum += n_ * (n_ - 1) / 2 * (x / m), x %= m;
      if (y >= m) sum += n_ * (y / m), y %= m;
      const long long top = x * n_ + y;
      if (top < m) break;
      n_ = top / m, y = top % m;
      const long long t = m;
      m = x, x = t;
    }
    return sum;
  }
  // The sum of x >> s over x = 0 .. n - 1.
  static __device__ __forceinline__ long long floors(long long n, int s) {
    const long long q = n >> s;
    return (q * (q - 1) / 2 << s) + q * (n & ((1LL << s) - 1));
  }
  __device__ long long all() const { return items ? before(items - 1) + tiles(items - 1) + kLead : 0; }
  static __device__ __forceinline__ long long floor_div(long long a, long long b) { return a >= 0 ? a / b : -1; }
};

// What a CTA does of an item: key tiles j0 .. j1 - 1 of `tiles` for the tokens from row0 on.
struct Item {
  int row0, tokens;  // row of q of the first token, tokens (none: there is no item)
  int seen;          // tokens that it sees, less one; may be negative
  int len, kvh, b;
  int j0, j1;
  int n0, n1;  // key tiles of tiles 0 and 1 (both those of tile 0 where they share it)
  int twin;
  int slot;  // -1: the whole item; 0: begun by others, 1: begun here and unfinished
};
// Steps of tile x: key tiles step(0) .. step(count - 1); rounds: turns of both tiles.
struct Steps {
  int x, j0, count, rounds, keys, stride, offset;
  __device__ __forceinline__ Steps(const Item& t, int x_) : x(x_), j0(t.j0) {
    keys = t.j1 - t.j0;
    stride = t.twin ? 2 : 1, offset = t.twin ? x : 0;
    rounds = t.twin ? (keys + 1) / 2 : keys;
    count = t.twin ? (keys + 1 - x) / 2 : max(min((x ? t.n1 : t.n0) - t.j0, keys), 0);
  }
  __device__ __forceinline__ int at(int r) const { return stride * r + offset; }  // key tile, less j0
};

__device__ __forceinline__ void sts_u128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// The codes of a key's row at `src` to fp16 numbers code * s + lo in row `row` of an operand tile, whose first box has it at
// `dst`.  Eight lanes read eight different 16-byte columns of the banks, and write eight.  V's channels stay in the order (0,
// 4), (1, 5), (2, 6), (3, 7) of kv_values8: the output is put right at the end.
template <int D, bool kV>
__device__ __forceinline__ void convert_row(uint32_t src, uint32_t dst, int row, uint32_t s2, uint32_t lo2) {
  constexpr int kN = KvI4<D>::kRow / 16;
  const int turn = D == 128 ? row >> 1 : 0;
  const uint32_t x = (row & 7) << 4;
  uint4 next = lds_u128(src + 16 * (turn & (kN - 1)));
  // rolled up: this runs between others' long stretches of code and would be fetched anew each time
#pragma unroll 1
  for (int i = 0; i < kN; ++i) {
    const int c = (i + turn) & (kN - 1);
    const uint32_t to = dst + (c >> 1) * Cfg<D>::kBox, xc = x ^ ((c & 1) << 6);
    const uint32_t w[4] = {next.x, next.y, next.z, next.w};
    next = lds_u128(src + 16 * ((i + 1 + turn) & (kN - 1)));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t h[4];
      kv_values8(w[e], s2, lo2, h);
      if constexpr (kV)
        sts_u128(to + (xc ^ (e << 4)), h[0], h[1], h[2], h[3]);
      else
        sts_u128(to + (xc ^ (e << 4)), prmt(h[0], h[1], 0x5410), prmt(h[2], h[3], 0x5410), prmt(h[0], h[1], 0x7632),
                 prmt(h[2], h[3], 0x7632));
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_chunks_i4_kernel(const __grid_constant__ CUtensorMap tm_q, const Args a) {
  using C = Cfg<D>;
  using L = KvI4<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Item s_item[2];
  __shared__ int s_bad[2];             // [parity of the item] first key whose V row is not finite
  __shared__ float2 s_ml[2][kTile];    // [parity of the item] (m, l) of tile 1's half of a shared tile
  __shared__ long long s_sum[kThreads / 32], s_off;
  __shared__ int s_b;
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t qbar, qfree;                              // Q tiles landed; not read any more
  __shared__ uint64_t raw_full[C::kRaw], raw_empty[C::kRaw];    // blocks landed; read (4 warps)
  __shared__ uint64_t full[C::kSlots], empty[C::kSlots];        // K or V tile written (4 warps); used (both tiles)
  __shared__ uint64_t sbar[2], pbar[2];                         // [tile] S complete; P written (4 warps)
  __shared__ uint64_t obar[2], ofree[2];                        // [tile] O complete; O read (4 warps)
  __shared__ uint64_t sfree[2], pfree[2];                       // [tile] P beside S: S read (4 warps); P used
  __shared__ uint64_t half;                                     // tile 1's half of a shared tile is complete (4 warps)
  __shared__ uint64_t item_full[2], item_empty[2];
  __shared__ uint64_t turn[2];                                  // [tile] its products may be queued
  __shared__ uint64_t done;                                     // every product (both tiles)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    mbar_init(&qbar, 1), mbar_init(&qfree, 2), mbar_init(&done, 2), mbar_init(&half, 4);
    for (int s = 0; s < C::kRaw; ++s) mbar_init(&raw_full[s], 1), mbar_init(&raw_empty[s], 4);
    for (int s = 0; s < C::kSlots; ++s) mbar_init(&full[s], 4), mbar_init(&empty[s], 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&turn[x], 1), mbar_init(&sbar[x], 1), mbar_init(&pbar[x], 4), mbar_init(&obar[x], 1), mbar_init(&ofree[x], 4);
      mbar_init(&sfree[x], 4), mbar_init(&pfree[x], 1);
      mbar_init(&item_full[x], 1), mbar_init(&item_empty[x], 3 + 8 + 8);  // copy, product, conversion and softmax warps
    }
    fence_mbarrier_init();
    mbar_arrive(&turn[0]);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();  // everything before this line overlaps the end of the preceding kernel
  grid_dependents_launch();

  // ---- this CTA's range [w0, w1) of the key tiles of all items, in the order of sequences, their items, K/V heads ----
  long long total, w0, w1;
  {
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
      mine += Shape(a, kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, blockIdx.x == 0 ? a.err : nullptr)).all() * a.Hkv;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_sum[warp] = incl;
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      total += s_sum[w];
    }
    const long long quota = (total + gridDim.x - 1) / gridDim.x;
    w0 = min(quota * blockIdx.x, total), w1 = min(w0 + quota, total);
    long long at = incl - mine;
    if (at <= w0 && w0 < incl && per == 1)
      s_b = b0, s_off = w0 - at;
    else if (at <= w0 && w0 < incl)
      for (int b = b0; b < b1; ++b) {
        const long long n = Shape(a, kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, nullptr)).all() * a.Hkv;
        if (w0 < at + n) {
          s_b = b, s_off = w0 - at;
          break;
        }
        at += n;
      }
    __syncthreads();
  }
  const uint32_t tmem = tmem_slot;
  if (w0 >= w1) {  // nothing to do, as where all sequences have a few rows
    if (tid == 0) a.parts.begun[blockIdx.x] = make_int4(0, 0, 0, 0), a.parts.went_on[blockIdx.x] = 0;
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }

  if (warp >= kLoadWarp) {
    if (warp >= kConvWarp)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ---------------- Q, and the codes and parameters of K(0), V(0), K(1), V(1) .. ----------------
      if (lane == 0) tma_prefetch_desc(&tm_q);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_warp(bar, phase & 1)) {
          if (lane == 0) report_error(a.err, kErrTimeoutEmpty);
          ok = false;
        }
        return ok;
      };
      uint32_t n = 0, rs = 0, rp = 0;  // half tiles so far, the next one's slot and round
      int items = 0;
      for (int it = 0; wait(&item_full[it & 1], it >> 1); ++it) {
        const Item t = s_item[it & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[it & 1]);
        if (t.tokens == 0) break;
        if (!wait(&qfree, (it & 1) ^ 1)) break;
        ++items;
        if (lane == 0) {
          const bool two = !t.twin;
          const int rows = a.tokens * a.G;
          mbar_arrive_expect_tx(&qbar, (two ? 2 : 1) * rows * D * 2);
          for (int x = 0; x < (two ? 2 : 1); ++x)
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(smem + x * C::kTileBytes + b * C::kBox, &tm_q, &qbar, 64 * b, t.kvh * a.G, t.row0 + x * a.tokens);
        }
        // Lane i looks after block i of half a tile: where it is the first one of a page, or of the half, it copies what
        // follows of that page.  A block is 16 tokens' K and V; small copies cost as much as large ones, so they go together.
        const int blocks = (t.len - 1) / kKvBlock + 1;  // of a sequence without tokens, one that is not copied
        auto starts = [&](int h) {                      // blocks to copy from here on
          const int gb = h * (kHalf / kKvBlock) + lane, in = gb - (int)quot((uint32_t)gb, a.by_bpp) * a.bpp;
          return lane < kHalf / kKvBlock && h < 2 * t.j1 && gb < blocks && t.len > 0 && (lane == 0 || in == 0)
                     ? min(min(kHalf / kKvBlock - lane, a.bpp - in), blocks - gb)
                     : 0;
        };
        auto page_of = [&](int h) {
          const int gb = h * (kHalf / kKvBlock) + lane;
          return starts(h) ? a.table[(long long)t.b * a.width + quot((uint32_t)gb, a.by_bpp)] : 0;
        };
        int page = page_of(2 * t.j0);
        for (int h = 2 * t.j0; h < 2 * t.j1; ++h) {
          const int next = page_of(h + 1), gb = h * (kHalf / kKvBlock) + lane;
          int run = starts(h);
          if (run && (page < 0 || page >= a.pages)) {
            report_error(a.err, kErrBadIndex);
            run = 0;
          }
          const uint32_t bytes = run * L::kBytes, all = __reduce_add_sync(0xffffffffu, bytes);
          if (!wait(&raw_empty[rs], (rp & 1) ^ 1)) break;
          if (lane == 0) {
            if (all)
              mbar_arrive_expect_tx(&raw_full[rs], all);
            else
              mbar_arrive(&raw_full[rs]);
          }
          __syncwarp();
          if (run) {
            const int in = gb - (int)quot((uint32_t)gb, a.by_bpp) * a.bpp;
            bulk_load(smem_u32(smem + C::kOffRaw + rs * C::kRawBytes) + lane * L::kBytes,
                      a.cache + (((long long)page * a.Hkv + t.kvh) * a.bpp + in) * L::kBytes, bytes, &raw_full[rs]);
          }
          ++n;
          if (++rs == C::kRaw) rs = 0, ++rp;
          page = next;
        }
      }
      // copies that may still be in flight land before the kernel ends
      bool landed = true;
      for (int i = 0; i < C::kRaw && i < (int)n && landed; ++i) {
        if (rs == 0) rs = C::kRaw, --rp;
        --rs;
        landed = mbar_wait_warp(&raw_full[rs], rp & 1);
      }
      if (items > 0 && landed) landed = mbar_wait_warp(&qbar, (items - 1) & 1);
      if (!landed && lane == 0) report_error(a.err, kErrTimeoutDrain);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ---------------- the tensor cores' work: a warp per tile, taking turns ----------------
      const int x = warp - kMmaWarp;
      const bool leader = elect_one();
      const uint32_t idesc_s = umma_idesc_f16(kTile, kTile, 0, 0) | a.negate;
      constexpr uint32_t idesc_o = umma_idesc_f16(kTile, D, /*A from TMEM*/ 0, /*B MN-major*/ 1);
      const uint32_t ring_lo = smem_u32(smem + C::kOffRing) >> 4;
      const uint32_t ts = tmem + x * kTile, to = tmem + C::kColO + x * D, tp = tmem + C::kColP + x * C::kStrideP;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_warp(bar, phase & 1)) {
          if (leader) report_error(a.err, kErrTimeoutMma);
          ok = false;
        }
        return ok;
      };
      auto release = [&](uint64_t* bar, bool used) {  // when the products queued so far are complete; at once without any
        if (!leader) return;
        if (used)
          umma_commit(bar);
        else
          mbar_arrive(bar);
      };
      // K and V tiles are numbered through all items: K of key tile j0 + s of this one is base + 2 s, V the next
      uint32_t base = 0;
      auto slot = [&](uint32_t n) { return n % C::kSlots; };
      auto wait_full = [&](uint32_t n) { return wait(&full[slot(n)], (int)(n / C::kSlots)); };
      auto qk = [&](uint32_t q_desc, uint32_t n) {  // S = Q K^T
        const uint32_t bd = (1u << 16) + ring_lo + slot(n) * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = ((s >> 2) * C::kBox + (s & 3) * 32) >> 4;
            mma_ss(ts, q_desc + off, bd + off, idesc_s, s > 0);
          }
          umma_commit(&sbar[x]);
        }
      };
      auto pv = [&](uint32_t n, uint32_t acc) {  // O (+)= P V
        const uint32_t bd = ((uint32_t)(C::kBox >> 4) << 16) + ring_lo + slot(n) * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s) mma_ts(to, tp + s * 8, bd + ((s * 2048) >> 4), idesc_o, s > 0 ? 1u : acc);
        }
      };
      int pcount = 0, ocount = 0, turns = 0, scount = 0;  // phases of pbar, of obar / ofree, of turn; S so far
      bool take_turns = false;  // both tiles read the same keys, and P is written over S
      auto my_turn = [&]() { return !take_turns || wait(&turn[x], turns++); };
      auto pass = [&]() {
        if (take_turns && leader) mbar_arrive(&turn[x ^ 1]);
      };
      auto s_free = [&]() {  // S may be written: its softmax has read it, where P does not say so
        const bool r = !C::kBeside || scount == 0 || wait(&sfree[x], scount - 1);
        ++scount;
        return r;
      };
      for (int it = 0; wait(&item_full[it & 1], it >> 1); ++it) {
        const Item t = s_item[it & 1];
        __syncwarp();
        if (leader) mbar_arrive(&item_empty[it & 1]);
        if (t.tokens == 0) break;
        const Steps st(t, x);
        const uint32_t end = base + 2 * st.keys;
        const uint32_t q_desc = (1u << 16) + ((smem_u32(smem) + (t.twin ? 0 : x) * C::kTileBytes) >> 4);
        const bool twin = t.twin;
        take_turns = !C::kBeside && !twin;
        // K or V tile n is not needed any more; where each half of the CTA has key tiles of its own, for both
        auto free_tile = [&](uint32_t n, bool used) {
          release(&empty[slot(n)], used);
          if (twin) release(&empty[slot(n)], used);
        };
        // S of the first step; the S columns are free, since the products that read their last P come before
        bool next = st.count > 0;
        if (!wait(&qbar, it) || !my_turn() || (next && !s_free())) break;
        if (next || !twin) {
          const uint32_t k = base + 2 * st.at(0);
          if (!wait_full(k)) break;
          tc_fence_after_sync();
          if (next) qk(q_desc, k);
          free_tile(k, next);
        }
        pass();
        if (st.count <= 1) release(&qfree, next);
        for (int r = 0; r < st.rounds && ok; ++r) {
          const bool now = r < st.count, some = now || !twin;  // a tile with fewer steps releases what the other has
          next = r + 1 < st.count;
          const bool some_next = next || (!twin && r + 1 < st.rounds);
          const uint32_t v = base + 2 * st.at(r) + 1, k = base + 2 * st.at(r + 1);
          if (C::kBeside && some_next) {
            if (!wait_full(k) || (next && !s_free())) break;
            tc_fence_after_sync();
            if (next) qk(q_desc, k);
            free_tile(k, next);
          }
          if (some && !wait_full(v)) break;
          // where both tiles read the same keys, the next K is there by now; else what it waits for may come after this step
          if (!C::kBeside && !twin && some_next && !wait_full(k)) break;
          if (now) {
            if (!wait(&pbar[x], pcount++)) break;
            // the accumulator is taken over when the softmax warps have read that of the item before
            if (r == 0 && ocount > 0 && !wait(&ofree[x], ocount - 1)) break;
          }
          if (!my_turn()) break;
          tc_fence_after_sync();
          if (now) {
            pv(v, r > 0);
            if (C::kBeside) release(&pfree[x], true);
            if (!next) {
              release(&obar[x], true);
              ++ocount;
            }
          }
          if (some) free_tile(v, now);
          if (!C::kBeside && some_next) {
            if (twin) {
              if (!wait_full(k)) break;
              tc_fence_after_sync();
            }
            if (next) qk(q_desc, k);
            free_tile(k, next);
          }
          pass();
          if (r + 2 == st.count) release(&qfree, true);
        }
        base = end;
      }
      if (ok) {
        release(&done, true);
        wait(&done, 0);
      }
    } else if (warp == kNextWarp) {
      // ---------------- the items of this CTA ----------------
      int4 begun = make_int4(0, 0, 0, 0);
      int went_on = 0, it = 0;
      bool ok = true;
      auto put = [&](const Item& t) {
        if (!mbar_wait_warp(&item_empty[it & 1], ((it >> 1) & 1) ^ 1)) {
          if (lane == 0) report_error(a.err, kErrTimeoutEmpty);
          ok = false;
          return;
        }
        if (lane == 0) {
          s_item[it & 1] = t, s_bad[it & 1] = INT_MAX;
          mbar_arrive(&item_full[it & 1]);
        }
        ++it;
      };
      {
        int b = s_b, p, kvh, s;
        KvChunk c = kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, nullptr);
        Shape sh(a, c);
        {  // the last item that begins at s_off or before: 32 guesses at a time
          int lo = 0, hi = sh.items - 1;
          while (lo < hi) {
            const int g = lo + (int)(((long long)(hi - lo) * (lane + 1) + 31) / 32);
            const unsigned yes = __ballot_sync(0xffffffffu, sh.before(g) * a.Hkv <= s_off);
            const int cnt = __popc(yes);  // of ascending guesses, the first ones
            const int below = __shfl_sync(0xffffffffu, g, max(cnt - 1, 0)), above = __shfl_sync(0xffffffffu, g, min(cnt, 31));
            if (cnt < 32) hi = above - 1;
            if (cnt > 0) lo = below;
          }
          p = lo;
          const long long rest = s_off - sh.before(p) * a.Hkv;
          const int cost = sh.tiles(p) + kLead;
          kvh = (int)(rest / cost), s = (int)(rest % cost);
        }
        long long left = w1 - w0;
        while (left > 0 && ok) {
          const int tiles = sh.tiles(p), cost = tiles + kLead;
          const int take = (int)min((long long)(cost - s), left);
          const int r0 = max(s - kLead, 0), r1 = s + take - kLead;
          if (r1 > r0) {
            Item t;
            t.row0 = c.start + p * sh.A, t.tokens = sh.count(p), t.seen = c.first + p * sh.A, t.len = c.len, t.kvh = kvh, t.b = b;
            t.twin = sh.twin(p);
            t.j0 = r0, t.j1 = r1;
            t.n0 = t.twin ? tiles : max(t.seen + a.tokens - 1, 0) / kTile + 1, t.n1 = tiles;
            t.slot = r0 > 0 ? 0 : r1 < tiles ? 1 : -1;
            if (t.slot == 0) went_on = r1 == tiles ? 2 : 1;
            if (t.slot == 1) begun = make_int4(t.row0, t.tokens, t.seen, kvh);
            put(t);
          }
          left -= take, s = 0;
          if (++kvh == a.Hkv && left > 0) {
            kvh = 0;
            if (++p == sh.items) {
              p = 0;
              do {
                c = kv_chunk(a.cu, a.kv_lens, ++b, a.T, a.cap, nullptr);
              } while (c.rows <= a.few);
              sh = Shape(a, c);
            }
          }
        }
      }
      if (lane == 0) a.parts.begun[blockIdx.x] = begun, a.parts.went_on[blockIdx.x] = went_on;
      if (ok) {
        Item t = {};
        put(t);
      }
    } else {
      // ---------------- codes to fp16: two warps K, two V of every other half tile, a thread one key's row ----------------
      const int group = (warp - kConvWarp) >> 2, v = (warp & 3) >= 2, key_in = tid & (kHalf - 1);
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_warp(bar, phase & 1)) {
          if (lane == 0) report_error(a.err, kErrTimeoutFull);
          ok = false;
        }
        return ok;
      };
      uint32_t n = 0;  // tiles so far
      for (int it = 0; wait(&item_full[it & 1], it >> 1); ++it) {
        const int j0 = s_item[it & 1].j0, j1 = s_item[it & 1].j1, len = s_item[it & 1].len, tokens = s_item[it & 1].tokens;
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[it & 1]);
        if (tokens == 0) break;
        for (int j = j0; j < j1; ++j, ++n) {
          const int row = group * kHalf + key_in, key = j * kTile + row;
          const uint32_t tile = 2 * n + v, slot = tile % C::kSlots, half_n = 2 * n + group, rs = half_n % C::kRaw;
          if (!wait(&raw_full[rs], (int)(half_n / C::kRaw)) || !wait(&empty[slot], (int)(tile / C::kSlots) ^ 1)) break;
          const uint8_t* raw = smem + C::kOffRaw + rs * C::kRawBytes + key_in / kKvBlock * L::kBytes;
          const uint32_t src = smem_u32(raw) + (v ? L::kV : 0) + key_in % kKvBlock * L::kRow;
          const uint32_t dst = smem_u32(smem + C::kOffRing + slot * C::kTileBytes) + row * 128;
          uint32_t par = row < len - j * kTile ? *reinterpret_cast<const uint32_t*>(raw + (v ? L::kVp : L::kKp) + 4 * (key_in % kKvBlock)) : 0u;
          if (!kv_finite(par)) {
            if (v) atomicMin(&s_bad[it & 1], key);
            par = v ? 0u : 0x7fff7fffu;
          }
          const uint32_t s2 = prmt(par, 0, 0x1010), lo2 = prmt(par, 0, 0x3232);
          if (v)
            convert_row<D, true>(src, dst, row, s2, lo2);
          else
            convert_row<D, false>(src, dst, row, s2, lo2);
          if (kv_overflows(par)) {  // rare; of a NaN: no
            for (int i = 0; i < D / 8; ++i) {
              const uint32_t at = dst + (i >> 3) * C::kBox + (((i & 7) ^ (row & 7)) << 4);
              const uint4 x = lds_u128(at);
              sts_u128(at, kv_clamp2(x.x), kv_clamp2(x.y), kv_clamp2(x.z), kv_clamp2(x.w));
            }
          }
          fence_proxy_async_smem();  // the tile for the products, and the codes' reads before the next copy
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[slot]), mbar_arrive(&raw_empty[rs]);
        }
      }
    }
  } else {
    // ---------------- softmax and output of tile x: thread r owns row r ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2, row = tid & 127, tok = row / a.G, g = row - tok * a.G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * kTile + lanes, to = tmem + C::kColO + x * D + lanes;
    const uint32_t tp = tmem + C::kColP + x * C::kStrideP + lanes;
    const float c = a.scale_log2;
    const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    int scount = 0, ocount = 0, pcount = 0, hcount = 0;  // phases of sbar, obar, half; P so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      if (ok && !mbar_wait_warp(bar, phase & 1)) {
        if (lane == 0) report_error(a.err, kErrTimeoutMma);
        ok = false;
      }
      return ok;
    };
    for (int it = 0; wait(&item_full[it & 1], it >> 1); ++it) {
      const Item& t = s_item[it & 1];
      if (t.tokens == 0) break;
      const Steps st(t, x);
      const bool twin = t.twin;
      const int seen = t.seen + (twin ? 0 : x * a.tokens);  // last key that the tile's first token sees
      float m = kNoMax, l0 = 0.f, l1 = 0.f;                 // m: what is subtracted from the scaled scores
      for (int r = 0; r < st.count && wait(&sbar[x], scount++); ++r) {
        tc_fence_after_sync();
        const int key0 = (st.j0 + st.at(r)) * kTile;
        if (seen - key0 < kTile - 1) {  // some row sees less than the whole tile
          const int last = seen + tok - key0;
#pragma unroll 1
          for (int i = 0; i < kTile; i += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(ts + i, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (i + e > last) v[e] = 0xff800000u;
            tmem_st_32x32b_x32(ts + i, v);
          }
          tmem_st_wait();
        }
        auto row_max = [&]() {  // of the scaled scores, less kTop
          float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll 1
          for (int i = 0; i < kTile; i += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(ts + i, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              top0 = max3(top0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              top1 = max3(top1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
          }
          return __fsub_rn(__fmul_rn(fmaxf(top0, top1), c), kTop);
        };
        // Rows that ask for it take a new maximum: only those, so that a row's roundings do not depend on its neighbours.  Rows
        // with large scores have them scaled and rounded first.  Returns the factor for the scores.
        auto raise = [&](float top, bool more) {
          const float now = more ? fmaxf(m, top) : m, f = ex2(m - now);
          m = now;
          const bool large = fabsf(m) > kLarge;
          if (__any_sync(0xffffffffu, large)) {
#pragma unroll 1
            for (int i = 0; i < kTile; i += 32) {
              uint32_t v[32];
              tmem_ld_32x32b_x32(ts + i, v);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), large ? c : 1.f));
              tmem_st_32x32b_x32(ts + i, v);
            }
            tmem_st_wait();
          }
          l0 *= f, l1 *= f;
          if (r > 0) {
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(to + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st_32x32b_x32(to + i, o);
            }
          }
          return large ? 1.f : c;
        };
        // The weights, kept until their sum has said that none of them is too large for fp16.
        uint32_t w[4][16];
        float a0, a1;  // this step's sums
        auto weights = [&](float mul) {
          a0 = a1 = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(ts + 32 * i, v);
            tmem_ld_wait();
            float f[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
#pragma unroll
            for (int e = 0; e < 32; e += 2) fma2(f[e], f[e + 1], mul, -m);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = ex2(f[e]);
#pragma unroll
            for (int e = 0; e < 32; e += 2) add2(a0, a1, f[e], f[e + 1]), w[i][e / 2] = pack_h2(f[e], f[e + 1]);
          }
        };
        if (r == 0) m = fmaxf(row_max(), kNoMax);
        weights(c);
        const bool more = a0 + a1 > kMost || fabsf(m) > kLarge;
        if (__any_sync(0xffffffffu, more)) {
          if (C::kBeside && pcount > 0 && !wait(&pfree[x], pcount - 1)) break;  // O is that of the steps before
          tc_fence_after_sync();
          weights(raise(row_max(), more));
        }
        if constexpr (C::kBeside) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[x]);
          if (pcount > 0 && !wait(&pfree[x], pcount - 1)) break;  // the last P has been used
          ++pcount;
          tc_fence_after_sync();
        }
        l0 += a0, l1 += a1;
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_st_32x32b_x16(tp + 16 * i, w[i]);
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pbar[x]);
      }
      float l = l0 + l1;
      if (st.count > 0 && !wait(&obar[x], ocount++)) break;
      tc_fence_after_sync();
      const bool shared = twin && st.keys > 1;  // both halves have steps
      if (twin && x) {
        if (shared) {
          s_ml[it & 1][row] = make_float2(m, l);
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&half);
        }
      } else {
        float f0 = 1.f, f1 = 0.f;
        if (shared) {
          if (!wait(&half, hcount++)) break;
          tc_fence_after_sync();
          const float2 ml = s_ml[it & 1][row];
          const float now = fmaxf(m, ml.x);
          f0 = ex2(m - now), f1 = ex2(ml.x - now);
          m = now, l = l * f0 + ml.y * f1;
        }
        const int mine = (twin ? 0 : x * a.tokens) + tok;  // token of the item
        const bool there = tok < a.tokens && mine < t.tokens, whole = t.slot < 0;
        const int last = seen + tok;  // the last key that this row sees
        const bool nan = last >= s_bad[it & 1];
        const long long to_row = whole ? (long long)(t.row0 + mine) * a.Hq + t.kvh * a.G + g
                                       : ((long long)blockIdx.x * 2 + t.slot) * a.parts.rows + mine * a.G + g;
        const float inv = last < 0 ? 0.f : 1.f / l;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          if (st.count > 0) {
            tmem_ld_32x32b_x32(to + i, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (shared) {
            uint32_t o1[32];
            tmem_ld_32x32b_x32(to + D + i, o1);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
          }
          if (!there) continue;
          if (nan) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0x7fc00000u;
          }
          // channel k of eight stands in column 2 k of theirs (k < 4) or 2 k - 7
          auto at = [](int ch) { return (ch & ~7) + ((ch & 7) < 4 ? 2 * (ch & 7) : 2 * (ch & 7) - 7); };
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                h[e] = pack_h2(__uint_as_float(o[at(j + 2 * e)]) * inv, __uint_as_float(o[at(j + 2 * e + 1)]) * inv);
              st_global_32(a.out + to_row * D + i + j, h, sectors);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t h[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) h[e] = o[at(j + e)];
              st_global_32(a.parts.part + to_row * D + i + j, h, true);
            }
          }
        }
        if (there && whole && a.lse) a.lse[to_row] = last < 0 ? -INFINITY : (m + lg2(l)) * 0.6931471805599453f;
        if (there && !whole) a.parts.ml[to_row] = make_float2(m, l);
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (st.count > 0) mbar_arrive(&ofree[x]);
          if (shared) mbar_arrive(&ofree[1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[it & 1]);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Joins the parts of items that CTAs shared, in their order: up to kJoinBlocks blocks for each CTA of the kernel above and then
// one for each of those that took sequences of a few rows, a warp per row.  One pass over a row's parts, kAhead of them in flight
// at a time.  More of them, or more rows of a warp at once, cost more by their registers than they save: the next kernel's CTAs
// need all of an SM's (512 tokens behind 15872: 136.7 us, four rows at once 140.4; a block for every eight rows 149.5).
constexpr int kJoinWarps = 8, kJoinBlocks = 8, kAhead = 4;

struct JoinArgs {
  ChunkParts parts, few;
  int blocks, ctas, Hq, G;  // no blocks: there are only the second ones
  __half* out;
  float* lse;
};

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_chunks_join_kernel(const JoinArgs a) {
  constexpr int kPer = D / 32;  // channels per lane
  const bool few = (int)blockIdx.x >= a.ctas * a.blocks;
  const ChunkParts w{few ? a.few.begun : a.parts.begun, few ? a.few.went_on : a.parts.went_on, few ? a.few.ml : a.parts.ml,
                     few ? a.few.part : a.parts.part, few ? a.few.rows : a.parts.rows};
  const int c = few ? blockIdx.x - a.ctas * a.blocks : blockIdx.x / a.blocks, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int4 it = w.begun[c];
  int v = c + 1 + lane < a.ctas ? w.went_on[c + 1 + lane] : 2;
  const int rows = it.y * a.G, step = (few ? 1 : a.blocks) * kJoinWarps;
  int r = (few ? 0 : blockIdx.x - c * a.blocks) * kJoinWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  int n = 1;  // parts: slot 1 of CTA c, slot 0 of those behind it
  for (;;) {
    const unsigned stop = __ballot_sync(0xffffffffu, v != 1);
    if (stop) {
      n += __ffs(stop);
      break;
    }
    n += 32;
    v = c + n + lane < a.ctas ? w.went_on[c + n + lane] : 2;
  }
  for (; r < rows; r += step) {
    float m = kNoMax, l = 0.f, o[kPer] = {};
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      float2 ml[kAhead];
      float x[kAhead][kPer];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k;
        const long long at = ((long long)(c + i) * 2 + (i == 0)) * w.rows + r;
        ml[k] = make_float2(kNoMax, 0.f);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[k][e] = 0.f;
        if (i < n) {
          ml[k] = w.ml[at];
          const float* src = w.part + at * D + kPer * lane;
          if constexpr (kPer == 4)
            *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(src);
          else
            *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(src);
        }
      }
      float now = m;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) now = fmaxf(now, ml[k].x);
      const float old = ex2(m - now);
      m = now, l *= old;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] *= old;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const float f = ex2(ml[k].x - m);
        l += ml[k].y * f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] += x[k][e] * f;
      }
    }
    const int tok = r / a.G;
    const bool none = it.z + tok < 0;  // sees nothing
    const float inv = none ? 0.f : 1.f / l;
    const long long to = (long long)(it.x + tok) * a.Hq + it.w * a.G + (r - tok * a.G);
    uint32_t h[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) h[e] = pack_h2(o[2 * e] * inv, o[2 * e + 1] * inv);
    if constexpr (kPer == 4)
      reinterpret_cast<uint2*>(a.out + to * D)[lane] = make_uint2(h[0], h[1]);
    else
      reinterpret_cast<uint32_t*>(a.out + to * D)[lane] = h[0];
    if (a.lse && lane == 0) a.lse[to] = none ? -INFINITY : (m + lg2(l)) * 0.6931471805599453f;
  }
}

int part_rows(int T, int G) {
  const long long rows = (long long)T * G, most = 2 * (kTile / G) * G;
  return (int)(rows < most ? rows : most);
}

template <int D>
cudaError_t launch(const CUtensorMap* q, const Args& a, const StepArgs* few, const JoinArgs& j, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_chunks_i4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(j.ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (q) {
    e = cudaLaunchKernelEx(&cfg, attn_chunks_i4_kernel<D>, *q, a);
    if (e != cudaSuccess) return e;
  }
  if (few) {
    e = launch_attn_steps_i4(*few, D, j.ctas, s);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(j.ctas * (j.blocks + (few ? 1 : 0)), 1, 1);
  cfg.blockDim = dim3(32 * kJoinWarps, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_chunks_join_kernel<D>, j);
}

// The workspace from `at` on (32-byte aligned; nullptr: to learn its size): O first, then (m, l), then what the CTAs say.
size_t lay_out(uint8_t* at, int ctas, int rows, int D, ChunkParts* p) {
  const size_t n = 2 * (size_t)ctas * rows;
  p->part = reinterpret_cast<float*>(at);
  p->ml = reinterpret_cast<float2*>(at + n * D * 4);
  p->begun = reinterpret_cast<int4*>(at + n * (D * 4 + 8));
  p->went_on = reinterpret_cast<int*>(at + n * (D * 4 + 8) + ctas * 16);
  p->rows = rows;
  return (n * (D * 4 + 8) + ctas * 20 + 31) & ~(size_t)31;
}

int few_rows(int T, int G) {
  const long long rows = (long long)T * G;
  return (int)(rows < kFewRows ? rows : kFewRows);
}

}  // namespace

size_t attn_chunks_i4_workspace_bytes(int T, int, int Hq, int Hkv, int D) {
  ChunkParts p;
  const int G = Hq / Hkv, ctas = num_sms();
  return lay_out(nullptr, ctas, part_rows(T, G), D, &p) + lay_out(nullptr, ctas, few_rows(T, G), D, &p) + 32;
}

cudaError_t launch_attn_chunks_i4(const uint16_t* q, long long q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                                  long long pages, int ps, const int* table, int width, const int* cu, const int* kv_lens,
                                  int B, float scale, uint16_t* out, float* lse, void* workspace, unsigned* dev_err,
                                  cudaStream_t s, std::string* err) {
  const int G = Hq / Hkv, tokens = kTile / G, ctas = num_sms();
  // Sequences of a few rows of a K/V head get a kernel of their own, where there may be such: not if all rows are one sequence's and
  // too many.  Up to eight rows if that is what the sequences have on the average, or more than sixteen and so some have many and
  // others surely few; else, and where a token has more than eight heads, up to sixteen.  The lengths are on the device, so rows of
  // no sequence count too, and a few sequences are judged by all: 32 x 4 drafted tokens of 4 heads (16 rows) take 35 us with heads
  // of 64 and 55 with heads of 128, but 76 and 100 in a q of twice as many rows, where they go to 128-row tiles.
  const long long mean = ((long long)T * G + B - 1) / B;
  const int most = G > 8 || (mean > 8 && mean <= kFewRows) ? kFewRows : 8;
  const int few = B > 1 || T <= most / G ? most / G : 0;
  const bool others = T > few;
  CUtensorMap tq;
  if (others && !make_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q, D, Hq, T, (uint64_t)D * 2, (uint64_t)q_stride * 2, 64, G,
                              tokens, CU_TENSOR_MAP_SWIZZLE_128B, err))
    return cudaErrorInvalidValue;
  JoinArgs j;
  uint8_t* w = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~(uintptr_t)31);
  w += lay_out(w, ctas, part_rows(T, G), D, &j.parts);
  lay_out(w, ctas, few_rows(T, G), D, &j.few);
  const int blocks = (j.parts.rows + kJoinWarps - 1) / kJoinWarps;
  j.blocks = !others ? 0 : blocks < kJoinBlocks ? blocks : kJoinBlocks;
  j.ctas = ctas, j.Hq = Hq, j.G = G, j.out = reinterpret_cast<__half*>(out), j.lse = lse;
  // a scale of zero keeps a trace of itself, so that masked scores stay minus infinity
  const float mag = scale < 0.f ? -scale : scale, scale_log2 = (mag < 1e-30f ? 1e-30f : mag) * 1.4426950408889634f;
  const Args a{cu, kv_lens, B, T, Hq, Hkv, G, tokens, cache, (int)pages, ps / kKvBlock, fast_div(ps / kKvBlock), table, width,
               width * ps, scale_log2, scale < 0.f ? 1u << 13 : 0u, j.out, lse, j.parts, few, dev_err};
  const StepArgs sa{reinterpret_cast<const __half*>(q), q_stride, cu, kv_lens, B, T, Hq, Hkv, G, few, cache, (int)pages,
                    fast_div(ps / kKvBlock), table, width, width * ps, scale < 0.f ? -scale_log2 : scale_log2, j.out, lse, j.few,
                    dev_err};
  const CUtensorMap* tiles = others ? &tq : nullptr;
  const StepArgs* steps = few ? &sa : nullptr;
  return D == 128 ? launch<128>(tiles, a, steps, j, s) : launch<64>(tiles, a, steps, j, s);
}

}  // namespace wql
