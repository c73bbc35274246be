// kv_weights_i4.cu -- the attention weight that every cached token gets from packed chunks of rows, added to running sums:
//   weights[b, kvh, t] += sum over the rows r of sequence b that see t, and the query heads h of kvh's group, of
//                         exp(scale q[r, h] . k[t] - lse[r, h]),   k = code * s + lo, rounded to fp16.
//
// The sums run over rows, so the keys are the first operand of the products (tcgen05): 128 of them are the lanes of a tile in
// tensor memory, where eight warps put them as fp16 numbers, a thread its key's row (no shared memory, and K is read from
// memory once).  The products of a tile with up to 64 rows (token, query head) put each key's scores into its lane, so a thread
// turns the scores of one key into weights and adds them up in a register: no exchange at all.
//
// A unit is 256 keys of a K/V head, two tiles; a step a tile of rows for a unit.  One warp finds the units, looks up their pages
// and has TMA bring codes and rows of q into two rings, one issues the products, eight convert and eight add up weights.  The
// steps of all units are divided evenly over the CTAs, one per SM; sums of units that CTAs share go to the workspace, and a
// second kernel adds them in their order.  What is added to a sum is added by the memory: no load, one operation per sum and
// call, so the order of CTAs does not show.
#include <atomic>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kTile = 128, kUnit = 2 * kTile;  // keys of a tile in tensor memory, and of a unit
constexpr int kRows = 64;                      // rows of a step at most
// warps 0-7: weights, four for each tile; 8-15: conversion, likewise; 16: units and copies; 17: products; 18, 19: none
constexpr int kThreads = 640, kConvWarp = 8, kLoadWarp = 16, kMmaWarp = 17;
constexpr int kLead = 1;  // steps that stand for a unit's own cost
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kCodes = kUnit * KvI4<D>::kRow;                // K's codes of a unit,
  static constexpr int kKeyBytes = kCodes + kUnit / kKvBlock * 128;   // with the parameters of K and V
  static constexpr int kKeySlots = 6, kRowSlots = 4;
  static constexpr int kRowBytes = kRows * D * 2, kBox = kRows * 128;  // a tile of q, its boxes of 64 channels
  static constexpr int kSmem = kRowSlots * kRowBytes + kKeySlots * kKeyBytes + 1024;
  static_assert(kSmem <= 224 * 1024, "shared memory");
  // tensor memory: scores [tile][two in turn][kRows], then the keys [two units in turn][tile][D / 2]
  static constexpr int kColK = 4 * kRows;
  static_assert(kColK + 4 * (D / 2) <= 512, "tensor memory");
};

struct Args {
  int T, Hq, Hkv, G;
  int tokens, heads, two;  // of a step: tokens, heads of each; 1: the heads of a token take two steps, 0: one
  FastDiv by_heads;
  int pages, bpp;  // bpp: blocks of a page
  FastDiv by_bpp;
  const int* table;
  int width, cap;
  const int *cu, *kv_lens;
  int B;
  float scale_log2;
  const float* lse;
  float* weights;
  // the workspace: the unit that each CTA began and left unfinished {sequence, K/V head, unit of it, 1}, whether it went on
  // with one (1) and ended it (2), and the sums of both [CTA][0: of the one found begun, 1: of the one begun][kUnit]
  int4* begun;
  int* went_on;
  float* part;
  unsigned* err;
};

// Steps of the units of a sequence: unit u takes the row tiles from skip(u) on, those before see none of its keys.
struct Shape {
  int units, tiles, per;  // per: row tiles that a unit's keys fill as tokens (tokens divides kUnit)
  long long c;            // row tiles that the tokens before row 0 fill
  __device__ __forceinline__ Shape(const Args& a, const KvChunk& k) {
    units = k.rows > 0 && k.len > 0 ? (k.len - 1) / kUnit + 1 : 0;
    tiles = k.rows > 0 ? ((k.rows - 1) / a.tokens + 1) << a.two : 0;
    per = kUnit / a.tokens << a.two;
    c = (k.first >= 0 ? ((unsigned)k.first + a.tokens - 1) / a.tokens : -(long long)(-k.first / a.tokens)) * (1 + a.two);
  }
  __device__ __forceinline__ int skip(int u) const { return (int)max((long long)per * u - c, 0LL); }
  __device__ __forceinline__ long long before(int u) const {  // the cost of units 0 .. u - 1
    const long long u0 = c < 0 ? 0 : min(c / per + 1, (long long)u);  // units that skip nothing
    return (long long)u * (kLead + tiles) - (per * ((long long)u * (u - 1) - u0 * (u0 - 1)) / 2 - c * (u - u0));
  }
};

// What a CTA does of a unit: row tiles tile0 .. tile1 - 1 of n tokens; the last token that the first one sees; -1 as slot: all
// that there is, else the part's place.
struct Unit {
  int b, kvh, u, len;
  int first, n, tile0, tile1;  // no tiles: there is no unit any more
  int slot;
};

// Two fp32 at once: x, y = (x, y) * m + (a, b).
__device__ __forceinline__ void fma2v(float& x, float& y, float m, float a, float b) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %4};\n"
      " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(m), "f"(a), "f"(b));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_i4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_codes,
                         const __grid_constant__ CUtensorMap tm_par, const Args a) {
  using L = KvI4<D>;
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit[C::kKeySlots];
  __shared__ __align__(16) float s_z[C::kRowSlots][kRows];  // -lse of the rows, times log2 e
  __shared__ uint64_t kfull[C::kKeySlots], kempty[C::kKeySlots];  // codes landed; unit done (17 warps)
  __shared__ uint64_t qfull[C::kRowSlots], qempty[C::kRowSlots];  // rows landed; products and weights done (1 + 8)
  __shared__ uint64_t afull[2], aempty[2];                        // keys in tensor memory (8 warps); products of the unit done
  __shared__ uint64_t sfull[2][2], sempty[2][2];                  // [tile][turn] scores complete; read (4 warps)
  __shared__ uint64_t done;
  __shared__ uint32_t tmem_slot;
  __shared__ long long s_sum[kThreads / 32], s_off;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* q_tiles = smem;
  uint8_t* keys = smem + C::kRowSlots * C::kRowBytes;
  if (tid == 0) {
    for (int i = 0; i < C::kKeySlots; ++i) mbar_init(&kfull[i], 1), mbar_init(&kempty[i], 17);
    for (int i = 0; i < C::kRowSlots; ++i) mbar_init(&qfull[i], 1), mbar_init(&qempty[i], 9);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], 8), mbar_init(&aempty[i], 1);
      for (int x = 0; x < 2; ++x) mbar_init(&sfull[x][i], 1), mbar_init(&sempty[x][i], 4);
    }
    mbar_init(&done, 1);
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- this CTA's range [w0, w1) of the steps of all units, in the order of sequences, K/V heads, units ----
  long long w0, w1;
  {
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto all = [&](int b, unsigned* err) {
      const Shape s(a, kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, err));
      return s.before(s.units) * a.Hkv;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += all(b, blockIdx.x == 0 ? a.err : nullptr);
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
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      total += s_sum[w];
    }
    const long long quota = (total + gridDim.x - 1) / gridDim.x;
    w0 = min(quota * blockIdx.x, total), w1 = min(w0 + quota, total);
    long long at = incl - mine;
    if (at <= w0 && w0 < incl)
      for (int b = b0; b < b1; ++b) {
        const long long n = all(b, nullptr);
        if (w0 < at + n) {
          s_b = b, s_off = w0 - at;
          break;
        }
        at += n;
      }
    __syncthreads();
  }

  const uint32_t tmem = tmem_slot;

  // What all warps do with units: wait for the next one, release the last.
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (ok && !mbar_wait_warp(bar, phase & 1)) {
      if (lane == 0) report_error(a.err, kErrTimeoutFull);
      ok = false;
    }
    return ok;
  };
  auto rows_of = [&](const Unit& t, int tile) {
    return min(t.n - (tile >> a.two) * a.tokens, a.tokens) * min(a.heads, a.G - (tile & a.two) * a.heads);
  };

  if (warp == kLoadWarp) {
    // ---------------- units, codes, rows ----------------
    if (lane == 0) tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_codes), tma_prefetch_desc(&tm_par);
    constexpr int kBlocks = kUnit / kKvBlock;
    // where four blocks lie together, one copy brings them; else each block has a lane and a copy of its own
    const int each = a.bpp % 4 == 0 ? 4 : 1;
    const uint32_t bytes = each * (kKvBlock * L::kRow + 128);
    int4 begun = make_int4(0, 0, 0, 0);
    int went_on = 0;
    uint32_t n = 0, m = 0;  // units, tiles of rows so far
    if (w0 < w1) {
      int b = s_b, kvh, u, s;
      KvChunk k = kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, nullptr);
      Shape sh(a, k);
      {
        const long long head = sh.before(sh.units);
        kvh = (int)(s_off / head);
        const long long off = s_off - kvh * head;
        int lo = 0, hi = sh.units - 1;  // the last unit that begins at off or before
        while (lo < hi) {
          const int mid = lo + (hi - lo + 1) / 2;
          if (sh.before(mid) <= off)
            lo = mid;
          else
            hi = mid - 1;
        }
        u = lo, s = (int)(off - sh.before(u));
      }
      long long left = w1 - w0;
      int in_b = -1, in_h = -1, in_tile = -1;  // the tile of rows that was loaded last
      while (left > 0 && ok) {
        const int skip = sh.skip(u), cost = kLead + sh.tiles - skip, take = (int)min((long long)(cost - s), left);
        const int r0 = max(s - kLead, 0), r1 = s + take - kLead;  // row tiles, from skip on
        if (r1 > r0) {
          const uint32_t ks = n % C::kKeySlots;
          const int gb = u * kBlocks + lane * each, blocks = (k.len - 1) / kKvBlock + 1;
          bool there = lane * each < kBlocks && gb < blocks;
          const int pg = (int)quot((uint32_t)gb, a.by_bpp), page = there ? a.table[(long long)b * a.width + pg] : 0;
          if (there && (page < 0 || page >= a.pages)) {
            report_error(a.err, kErrBadIndex);
            there = false;
          }
          if (!wait(&kempty[ks], n / C::kKeySlots ^ 1)) break;
          const uint32_t all = __popc(__ballot_sync(0xffffffffu, there)) * bytes;
          if (lane == 0) {
            Unit& t = s_unit[ks];
            t.b = b, t.kvh = kvh, t.u = u, t.len = k.len, t.first = k.first, t.n = k.rows;
            t.tile0 = skip + r0, t.tile1 = skip + r1;
            t.slot = r0 > 0 ? 0 : r1 + kLead < cost ? 1 : -1;
            if (all)
              mbar_arrive_expect_tx(&kfull[ks], all);
            else
              mbar_arrive(&kfull[ks]);
          }
          __syncwarp();
          if (there) {
            const int block = (int)(((long long)page * a.Hkv + kvh) * a.bpp + (gb - pg * a.bpp));
            uint8_t* dst = keys + ks * C::kKeyBytes;
            tma_load_3d(dst + lane * each * kKvBlock * L::kRow, &tm_codes, &kfull[ks], 0, 0, block);
            tma_load_3d(dst + C::kCodes + lane * each * 128, &tm_par, &kfull[ks], 0, L::kKp / 128, block);
          }
          ++n;
          if (r0 > 0) went_on = r1 + kLead == cost ? 2 : 1;
          else if (r1 + kLead < cost) begun = make_int4(b, kvh, u, 1);
          for (int tile = skip + r0; tile < skip + r1; ++tile) {
            if (in_b == b && in_h == kvh && in_tile == tile) continue;
            in_b = b, in_h = kvh, in_tile = tile;
            const uint32_t qs = m % C::kRowSlots;
            const int t0 = (tile >> a.two) * a.tokens, h0 = kvh * a.G + (tile & a.two) * a.heads;
            // the rows' lse, in registers before the slot is waited for
            float z[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = 32 * i + lane, tok = (int)quot((uint32_t)row, a.by_heads), h = h0 + row - tok * a.heads;
              z[i] = tok < a.tokens && t0 + tok < k.rows && h < a.Hq ? a.lse[(long long)(k.start + t0 + tok) * a.Hq + h] * -kLog2e
                                                                     : 0.f;
            }
            if (!wait(&qempty[qs], m / C::kRowSlots ^ 1)) break;
            s_z[qs][lane] = z[0], s_z[qs][32 + lane] = z[1];
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_expect_tx(&qfull[qs], a.tokens * a.heads * D * 2);
              for (int i = 0; i < D / 64; ++i)
                tma_load_3d(q_tiles + qs * C::kRowBytes + i * C::kBox, &tm_q, &qfull[qs], 64 * i, h0, k.start + t0);
            }
            ++m;
          }
        }
        left -= take, s = 0;
        if (left > 0 && ++u == sh.units) {
          u = 0;
          if (++kvh == a.Hkv) {
            kvh = 0;
            do {
              k = kv_chunk(a.cu, a.kv_lens, ++b, a.T, a.cap, nullptr);
              sh = Shape(a, k);
            } while (sh.units == 0);
          }
        }
      }
    }
    if (lane == 0) a.begun[blockIdx.x] = begun, a.went_on[blockIdx.x] = went_on;
    if (wait(&kempty[n % C::kKeySlots], n / C::kKeySlots ^ 1) && lane == 0) {
      s_unit[n % C::kKeySlots].tile1 = s_unit[n % C::kKeySlots].tile0 = 0;
      mbar_arrive(&kfull[n % C::kKeySlots]);
    }
    // copies that may still be in flight land before the kernel ends; what was in the slot of the end has been read
    bool landed = true;
    for (int i = 0; i < C::kKeySlots - 1 && n > 0 && landed; ++i) {
      --n;
      landed = mbar_wait_warp(&kfull[n % C::kKeySlots], n / C::kKeySlots & 1);
    }
    for (int i = 0; i < C::kRowSlots && m > 0 && landed; ++i) {
      --m;
      landed = mbar_wait_warp(&qfull[m % C::kRowSlots], m / C::kRowSlots & 1);
    }
    if (!landed && lane == 0) report_error(a.err, kErrTimeoutDrain);
  } else if (warp == kMmaWarp) {
    // ---------------- products ----------------
    const bool leader = elect_one();
    const uint32_t q_lo = (1u << 16) + (smem_u32(q_tiles) >> 4);
    uint32_t m = 0, steps = 0;
    int in_b = -1, in_h = -1, in_tile = -1;
    for (uint32_t n = 0; wait(&kfull[n % C::kKeySlots], n / C::kKeySlots); ++n) {
      const Unit t = s_unit[n % C::kKeySlots];
      __syncwarp();
      if (leader) mbar_arrive(&kempty[n % C::kKeySlots]);
      if (t.tile0 == t.tile1 || !wait(&afull[n & 1], n >> 1)) break;
      tc_fence_after_sync();
      for (int tile = t.tile0; tile < t.tile1; ++tile, ++steps) {
        if (in_b != t.b || in_h != t.kvh || in_tile != tile) {  // as the copies go: another tile of rows
          in_b = t.b, in_h = t.kvh, in_tile = tile;
          if (m > 0 && leader) umma_commit(&qempty[(m - 1) % C::kRowSlots]);
          if (!wait(&qfull[m % C::kRowSlots], m / C::kRowSlots)) break;
          ++m;
        }
        const uint32_t bd = q_lo + (m - 1) % C::kRowSlots * (C::kRowBytes >> 4), turn = steps & 1;
        const uint32_t idesc = umma_idesc_f16(kTile, (rows_of(t, tile) + 15) & ~15, 0, 0);
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (!wait(&sempty[x][turn], (steps >> 1) ^ 1)) break;
          tc_fence_after_sync();
          if (leader) {
            const uint32_t d = tmem + (2 * x + turn) * kRows, ak = tmem + C::kColK + (2 * (n & 1) + x) * (D / 2);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_ts(d, ak + 8 * s, bd + (((s >> 2) * C::kBox + (s & 3) * 32) >> 4), idesc, s > 0);
            umma_commit(&sfull[x][turn]);
          }
        }
      }
      if (leader) umma_commit(&aempty[n & 1]);
    }
    if (ok) {
      if (leader) umma_commit(&done);
      wait(&done, 0);
    }
  } else if (warp >= kConvWarp && warp < kLoadWarp) {
    // ---------------- codes to fp16: a thread takes one key's row, a lane of tensor memory ----------------
    const int x = (warp - kConvWarp) >> 2, row = (tid - 32 * kConvWarp) & (kUnit - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    for (uint32_t n = 0; wait(&kfull[n % C::kKeySlots], n / C::kKeySlots); ++n) {
      const uint32_t ks = n % C::kKeySlots;
      const bool end = s_unit[ks].tile0 == s_unit[ks].tile1, inside = row < s_unit[ks].len - s_unit[ks].u * kUnit;
      if (end || !wait(&aempty[n & 1], (n >> 1) ^ 1)) break;
      tc_fence_after_sync();
      const uint32_t raw = smem_u32(keys + ks * C::kKeyBytes);
      uint32_t p = lds_u32(raw + C::kCodes + row / kKvBlock * 128 + row % kKvBlock * 4);
      if (!inside) p = 0u;
      if (!kv_finite(p)) p = 0x7fff7fffu;
      const uint32_t s2 = prmt(p, 0, 0x1010), lo2 = prmt(p, 0, 0x3232);
      const uint32_t to = tmem + C::kColK + (2 * (n & 1) + x) * (D / 2) + lanes;
      auto convert = [&](auto clamp) {
#pragma unroll 1
        for (int i = 0; i < L::kRow / 16; ++i) {
          // heads of 128: two keys' codes to a line of 128 bytes, swizzled, so that lanes that read together meet no bank twice
          const uint4 v = lds_u128(D == 128 ? raw + (row >> 1) * 128 + ((((row & 1) * 4 + i) ^ ((row >> 1) & 7)) << 4)
                                            : raw + row * L::kRow + 16 * i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[4];
            kv_values8(w[e], s2, lo2, h);
            o[4 * e] = prmt(h[0], h[1], 0x5410), o[4 * e + 1] = prmt(h[2], h[3], 0x5410);
            o[4 * e + 2] = prmt(h[0], h[1], 0x7632), o[4 * e + 3] = prmt(h[2], h[3], 0x7632);
          }
          if constexpr (decltype(clamp)::value) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = kv_clamp2(o[e]);
          }
          tmem_st_32x32b_x16(to + 16 * i, o);
        }
      };
      if (__any_sync(0xffffffffu, kv_overflows(p)))  // rare; of a NaN: no
        convert(std::true_type());
      else
        convert(std::false_type());
      fence_proxy_async_smem();  // these reads come before the copies that follow them into the slot
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&afull[n & 1]), mbar_arrive(&kempty[ks]);
    }
  } else if (warp < kConvWarp) {
    // ---------------- weights: a thread takes one key ----------------
    const int x = warp >> 2, row = tid & (kUnit - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t m = 0, steps = 0;
    int in_b = -1, in_h = -1, in_tile = -1;
    for (uint32_t n = 0; wait(&kfull[n % C::kKeySlots], n / C::kKeySlots); ++n) {
      const Unit t = s_unit[n % C::kKeySlots];
      __syncwarp();
      if (lane == 0) mbar_arrive(&kempty[n % C::kKeySlots]);
      if (t.tile0 == t.tile1) break;
      const int key0 = t.u * kUnit;
      float sum[4] = {};
      for (int tile = t.tile0; tile < t.tile1; ++tile, ++steps) {
        if (in_b != t.b || in_h != t.kvh || in_tile != tile) {
          in_b = t.b, in_h = t.kvh, in_tile = tile;
          if (m > 0 && lane == 0) mbar_arrive(&qempty[(m - 1) % C::kRowSlots]);
          if (!wait(&qfull[m % C::kRowSlots], m / C::kRowSlots)) break;  // for s_z
          ++m;
        }
        const float* z = s_z[(m - 1) % C::kRowSlots];
        const uint32_t turn = steps & 1, from = tmem + (2 * x + turn) * kRows + lanes;
        const int rows = rows_of(t, tile), first = t.first + (tile >> a.two) * a.tokens;
        if (!wait(&sfull[x][turn], steps >> 1)) break;
        tc_fence_after_sync();
        auto add = [&](const uint32_t (&v)[32], int col, int lo, int hi, auto careful) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (decltype(careful)::value && e >= hi) break;
            const float4 z4 = *reinterpret_cast<const float4*>(z + col + e);
            float p0 = __uint_as_float(v[e]), p1 = __uint_as_float(v[e + 1]), p2 = __uint_as_float(v[e + 2]),
                  p3 = __uint_as_float(v[e + 3]);
            fma2v(p0, p1, a.scale_log2, z4.x, z4.y);
            fma2v(p2, p3, a.scale_log2, z4.z, z4.w);
            p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
            if constexpr (decltype(careful)::value) {
              p0 = e >= lo && e < hi ? p0 : 0.f, p1 = e + 1 >= lo && e + 1 < hi ? p1 : 0.f;
              p2 = e + 2 >= lo && e + 2 < hi ? p2 : 0.f, p3 = e + 3 >= lo && e + 3 < hi ? p3 : 0.f;
            }
            add2(sum[0], sum[1], p0, p1);
            add2(sum[2], sum[3], p2, p3);
          }
        };
        uint32_t v0[32], v1[32];
        tmem_ld_32x32b_x32(from, v0);
        tmem_ld_wait();
        if (rows > 32) tmem_ld_32x32b_x32(from + 32, v1);
        // columns [lo, rows) are rows that see this key
        const int lo = min(max(key0 - first + row, 0), kRows) * a.heads;
        if (key0 - first + (row | 31) > 0 || rows % 32 != 0) {
          add(v0, 0, lo, rows, std::true_type());
          tmem_ld_wait();
          if (rows > 32) add(v1, 32, lo - 32, rows - 32, std::true_type());
        } else {
          add(v0, 0, 0, 32, std::false_type());
          tmem_ld_wait();
          if (rows > 32) add(v1, 32, 0, 32, std::false_type());
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[x][turn]);
      }
      const float mine = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (t.slot >= 0)
        a.part[((long long)blockIdx.x * 2 + t.slot) * kUnit + row] = mine;
      else if (row < t.len - key0)
        atomicAdd(a.weights + ((long long)t.b * a.Hkv + t.kvh) * a.cap + key0 + row, mine);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// Adds the sums of the unit that CTA blockIdx.x began and others went on with.
__global__ void __launch_bounds__(kUnit) kv_weights_join_kernel(const Args a, int ctas) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int c = blockIdx.x;
  const int4 it = a.begun[c];
  if (it.w == 0) return;
  float sum = a.part[((long long)c * 2 + 1) * kUnit + threadIdx.x];
  for (int i = c + 1; i < ctas; ++i) {
    const int v = a.went_on[i];
    sum += a.part[(long long)i * 2 * kUnit + threadIdx.x];
    if (v != 1) break;
  }
  if ((int)threadIdx.x < min(max(a.kv_lens[it.x], 0), a.cap) - it.z * kUnit)
    a.weights[((long long)it.x * a.Hkv + it.y) * a.cap + it.z * kUnit + threadIdx.x] += sum;
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& codes, const CUtensorMap& par, const Args& a, int ctas,
                   cudaStream_t s) {
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_weights_i4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_weights_i4_kernel<D>, q, codes, par, a);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kUnit, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_weights_join_kernel, a, ctas);
}

}  // namespace

size_t kv_weights_i4_workspace_bytes() { return (size_t)num_sms() * (2 * kUnit * 4 + 32); }

cudaError_t launch_kv_weights_i4(const uint16_t* q, long long q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                                 long long pages, int ps, const int* table, int width, const int* cu, const int* kv_lens, int B,
                                 float scale, const float* lse, float* weights, void* workspace, unsigned* dev_err,
                                 cudaStream_t s, std::string* err) {
  const int ctas = num_sms(), G = Hq / Hkv;
  // a step: as many tokens as fit, a power of two, which divides kUnit; where a token has more heads, they take two steps
  const int heads = G < kRows ? G : kRows;
  int tokens = 1;
  while (2 * tokens * heads <= kRows) tokens *= 2;
  const uint64_t piece = 128, block = kKvBlock * (D + 8), blocks = (uint64_t)pages * Hkv * (ps / kKvBlock);
  const uint32_t together = ps % 64 == 0 ? 4 : 1;
  CUtensorMap tq, tc, tp;
  if (!make_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q, D, Hq, T, (uint64_t)D * 2, (uint64_t)q_stride * 2, 64, heads, tokens,
                    CU_TENSOR_MAP_SWIZZLE_128B, err) ||
      !make_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, piece, block / piece, blocks, piece, block, piece,
                    kKvBlock * D / 2 / piece, together, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    err) ||
      !make_tmap_3d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, piece, block / piece, blocks, piece, block, piece, 1, together,
                    CU_TENSOR_MAP_SWIZZLE_NONE, err))
    return cudaErrorInvalidValue;
  float* part = static_cast<float*>(workspace);
  int4* begun = reinterpret_cast<int4*>(part + (size_t)ctas * 2 * kUnit);
  Args a{T, Hq, Hkv, G, tokens, heads, G > kRows, fast_div(heads), (int)pages, ps / kKvBlock, fast_div(ps / kKvBlock), table, width,
         width * ps, cu, kv_lens, B, scale * kLog2e, lse, weights, begun,
         reinterpret_cast<int*>(begun + ctas), part, dev_err};
  return D == 128 ? launch<128>(tq, tc, tp, a, ctas, s) : launch<64>(tq, tc, tp, a, ctas, s);
}

}  // namespace wql
