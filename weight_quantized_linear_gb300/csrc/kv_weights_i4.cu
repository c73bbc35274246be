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
// and has TMA bring codes and rows of q into two rings, two issue the products, and of three groups of eight some convert and
// some add up weights, as the rows at hand ask.  The steps of all units are divided evenly over the CTAs, one per SM; sums of units
// that CTAs share go to the workspace, and a second kernel adds them in their order.  What is added to a sum is added by the memory:
// no load, one operation per sum and call, so the order of CTAs does not show.
//
// Bound, with many rows, by the exponentials and what surrounds them: a step of 64 rows and 256 keys is 512 cycles of the units for
// those and takes 1150 (issue slots 66 % used, 40 % of them for exponentials); with few rows by the conversion and the one warp that
// brings codes, 2300 cycles per unit, at 31 % of the memory's rate.  One row of a product is one weight in one lane, so nothing is
// exchanged; the first kernel, mma.sync with K in registers, took 38, 81 and 298 us for the figures below.
// Measured on GB300 through the Python call:
//   the last 32 tokens over 32768, 32 / 8 heads of 128          24 us, in a graph as well (the call's host time, beside it: 26)
//   64 single tokens over up to 8192, 32 / 8 heads of 128       78 us, 2.1 TB/s
//   whole prompts up to 4099 tokens, 32 / 8 heads of 64        194 us, 382 TFLOP/s
//
// Roundings: the difference of score and lse is formed in one fp32 operation, the exponential is the GPU's approximation to base 2
// (2^-22), sums are fp32.  Weights of whole prompts are off by 2e-7 of themselves, as fp32 scores are; an exact exponential would take
// several times the one operation that bounds this kernel.
#include <atomic>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kTile = 128, kUnitLog2 = 8, kUnit = 2 * kTile;  // keys of a tile in tensor memory, and of a unit
constexpr int kRows = 64;                      // rows of a step at most
// Warps work in groups of eight, four for each tile: groups that add up weights take steps in turn, groups that convert take
// units in turn, and four single warps follow: units and copies, products of each tile, none.
constexpr int kGroups = 3, kThreads = 32 * (8 * kGroups + 4), kLoadWarp = 8 * kGroups, kMmaWarp = kLoadWarp + 1;
// registers per thread: launched with 72, two warpgroups of those that convert give 8 each at least
constexpr int kConvRegs = 64, kLoadRegs = 80;
constexpr int kLead = 1;  // steps that stand for a unit's own cost
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int kSoft>  // kSoft: groups that add up weights; the others convert
struct Cfg {
  static constexpr int kConv = kGroups - kSoft;
  // with few rows a tile of them serves many units in turn; with many, each step has a slot of its own
  static constexpr bool kReuse = kSoft == 1;
  static constexpr int kCodes = kUnit * KvI4<D>::kRow;                // K's codes of a unit,
  static constexpr int kKeyBytes = kCodes + kUnit / kKvBlock * 128;   // with the parameters of K and V
  static constexpr int kKeySlots = 6, kRowSlots = 4;
  // Groups that take turns meet every phase of a barrier only if turns and slots go round together; else one could take an old
  // phase for the next.  Rows' slots are waited for by warps that take them all.
  static_assert(kKeySlots % kConv == 0 && 2 % kConv == 0, "key slots, and keys in tensor memory: one converting group's each");
  static_assert(2 % kSoft == 0, "the two places for scores: one adding group's each");
  static constexpr int kRowBytes = kRows * D * 2, kBox = kRows * 128;  // a tile of q, its boxes of 64 channels
  static constexpr int kSmem = kRowSlots * kRowBytes + kKeySlots * kKeyBytes + 1024;
  static_assert(kSmem <= 224 * 1024, "shared memory");
  // tensor memory: scores [tile][two in turn][kRows], then the keys [two units in turn][tile][D / 2]
  static constexpr int kColK = 4 * kRows;
  static_assert(kColK + 4 * (D / 2) <= 512, "tensor memory");
};

struct Args {
  int T, Hq, Hkv, G;
  int tokens_log2, tokens, heads, two;  // of a step: tokens, heads of each; 1: the heads of a token take two steps, 0: one
  FastDiv by_heads;
  int pages, bpp;  // bpp: blocks of a page
  FastDiv by_bpp;
  const int* table;
  int width, cap;
  const int *cu, *kv_lens;
  int B;
  float scale;
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
  int units, tiles, per;  // per: log2 of the row tiles that a unit's keys fill as tokens
  long long c;            // row tiles that the tokens before row 0 fill
  __device__ __forceinline__ Shape(const Args& a, const KvChunk& k) {
    units = k.rows > 0 && k.len > 0 ? (k.len - 1) / kUnit + 1 : 0;
    tiles = k.rows > 0 ? (((k.rows - 1) >> a.tokens_log2) + 1) << a.two : 0;
    per = kUnitLog2 - a.tokens_log2 + a.two;
    c = (((long long)k.first + a.tokens - 1) >> a.tokens_log2) * (1 + a.two);
  }
  __device__ __forceinline__ int skip(int u) const { return (int)max(((long long)u << per) - c, 0LL); }
  __device__ __forceinline__ long long before(int u) const {  // the cost of units 0 .. u - 1
    const long long u0 = c < 0 ? 0 : min((c >> per) + 1, (long long)u);  // units that skip nothing
    return (long long)u * (kLead + tiles) - ((((long long)u * (u - 1) - u0 * (u0 - 1)) / 2 << per) - c * (u - u0));
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

__device__ __forceinline__ void mul2(float& x, float& y, float m) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mul.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(m));
}
// Four bytes to shared memory without waiting for them, and an arrival on `bar` once this thread's have landed.
__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

template <int D, int kSoft>
__global__ void __launch_bounds__(kThreads, 1)
    kv_weights_i4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_codes,
                         const __grid_constant__ CUtensorMap tm_par, const Args a) {
  using L = KvI4<D>;
  using C = Cfg<D, kSoft>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit[C::kKeySlots];
  __shared__ __align__(16) float s_z[C::kRowSlots][kRows];  // lse of the rows
  __shared__ float s_other[2][kUnit];                       // [unit in turn] what the second group adds to the first's sums
  __shared__ uint64_t kfull[C::kKeySlots], kempty[C::kKeySlots];  // codes landed; unit read (groups of 8, products)
  __shared__ uint64_t qfull[C::kRowSlots], qempty[C::kRowSlots];  // rows and their lse landed; used
  __shared__ uint64_t afull[2], aempty[2];                        // keys in tensor memory (8 warps); products of the unit done
  __shared__ uint64_t ofull[2], oempty[2];                        // s_other written, read (8 warps)
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
    for (int i = 0; i < C::kKeySlots; ++i) mbar_init(&kfull[i], 1), mbar_init(&kempty[i], 8 + 2 + 8 * kSoft);
    for (int i = 0; i < C::kRowSlots; ++i) mbar_init(&qfull[i], 1 + 32), mbar_init(&qempty[i], 2 + 8);  // the products of both tiles, a group
    for (int i = 0; i < 2; ++i) {
      mbar_init(&afull[i], 8), mbar_init(&aempty[i], 2), mbar_init(&ofull[i], 8), mbar_init(&oempty[i], 8);
      for (int x = 0; x < 2; ++x) mbar_init(&sfull[x][i], 1), mbar_init(&sempty[x][i], 4);
    }
    mbar_init(&done, 2);
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
    if (at <= w0 && w0 < incl && per == 1)
      s_b = b0, s_off = w0 - at;
    else if (at <= w0 && w0 < incl)
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
  if (warp >= kLoadWarp)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
  else if (warp >= 8 * kSoft)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));

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
        int lo = 0, hi = sh.units - 1;  // the last unit that begins at off or before: 32 guesses at a time
        while (lo < hi) {
          const int guess = lo + (int)(((long long)(hi - lo) * (lane + 1) + 31) / 32);
          const int cnt = __popc(__ballot_sync(0xffffffffu, sh.before(guess) <= off));  // of ascending guesses, the first ones
          const int below = __shfl_sync(0xffffffffu, guess, max(cnt - 1, 0)), above = __shfl_sync(0xffffffffu, guess, min(cnt, 31));
          if (cnt < 32) hi = above - 1;
          if (cnt > 0) lo = below;
        }
        u = lo, s = (int)(off - sh.before(u));
      }
      // Pages are looked up for 32 copies at a time, and those of the next 32 with them: this warp's round has to be shorter
      // than a load.  The heads of a sequence begin with the same ones.
      const int lanes = kBlocks / each, per = 32 / lanes;  // of a unit; units
      auto look_up = [&](int u_) {
        const int gb = u_ * kBlocks + lane * each;
        return gb < (k.len - 1) / kKvBlock + 1 ? a.table[(long long)b * a.width + quot((uint32_t)gb, a.by_bpp)] : 0;
      };
      int page0 = look_up(0), page_next = look_up(u), page_u = u - per;
      int block = -1;  // of this lane's copy; -1: none
      auto take_pages = [&](int page, int u_) {
        const int gb = u_ * kBlocks + lane * each;
        const bool inside = gb < (k.len - 1) / kKvBlock + 1, good = page >= 0 && page < a.pages;
        if (inside && !good) report_error(a.err, kErrBadIndex);
        block = inside && good ? (int)(((long long)page * a.Hkv + kvh) * a.bpp + (gb - (int)quot((uint32_t)gb, a.by_bpp) * a.bpp)) : -1;
        page_u = u_, page_next = look_up(u_ + per);
      };
      const int tok0 = (int)quot((uint32_t)lane, a.by_heads), tok1 = (int)quot((uint32_t)lane + 32, a.by_heads);
      const int at0 = tok0 * a.Hq + (lane - tok0 * a.heads), at1 = tok1 * a.Hq + (lane + 32 - tok1 * a.heads);
      long long left = w1 - w0;
      int in_b = -1, in_h = -1, in_tile = -1;  // the tile of rows that was loaded last
      while (left > 0 && ok) {
        const int skip = sh.skip(u), cost = kLead + sh.tiles - skip, take = (int)min((long long)(cost - s), left);
        const int r0 = max(s - kLead, 0), r1 = s + take - kLead;  // row tiles, from skip on
        if (r1 > r0) {
          const uint32_t ks = n % C::kKeySlots;
          if (u == 0)
            take_pages(page0, 0);
          else if (u == page_u + per)
            take_pages(page_next, u);
          const int sub = lane - (u - page_u) * lanes;
          const bool there = sub >= 0 && sub < lanes && block >= 0;
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
            uint8_t* dst = keys + ks * C::kKeyBytes;
            tma_load_3d(dst + sub * each * kKvBlock * L::kRow, &tm_codes, &kfull[ks], 0, 0, block);
            tma_load_3d(dst + C::kCodes + sub * each * 128, &tm_par, &kfull[ks], 0, L::kKp / 128, block);
          }
          ++n;
          if (r0 > 0) went_on = r1 + kLead == cost ? 2 : 1;
          else if (r1 + kLead < cost) begun = make_int4(b, kvh, u, 1);
          for (int tile = skip + r0; tile < skip + r1; ++tile) {
            if (C::kReuse && in_b == b && in_h == kvh && in_tile == tile) continue;
            in_b = b, in_h = kvh, in_tile = tile;
            const uint32_t qs = m % C::kRowSlots;
            const int t0 = (tile >> a.two) * a.tokens, h0 = kvh * a.G + (tile & a.two) * a.heads, some = min(k.rows - t0, a.tokens);
            if (!wait(&qempty[qs], m / C::kRowSlots ^ 1)) break;
            // nothing here waits for a load: what is not a row of this step keeps a value that nobody takes
            const float* z = a.lse + (long long)(k.start + t0) * a.Hq + h0;
            const int most = a.Hq - h0;  // heads
            if (tok0 < some && at0 - tok0 * a.Hq < most) cp_async_4(&s_z[qs][lane], z + at0);
            if (tok1 < some && at1 - tok1 * a.Hq < most) cp_async_4(&s_z[qs][32 + lane], z + at1);
            cp_async_arrive(&qfull[qs]);
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
            page0 = look_up(0);
          }
        }
      }
    }
    if (lane == 0) a.begun[blockIdx.x] = begun, a.went_on[blockIdx.x] = went_on;
    // copies that may still be in flight land before the kernel ends
    bool landed = true;
    for (uint32_t i = 1; i <= C::kKeySlots && i <= n && landed; ++i)
      landed = mbar_wait_warp(&kfull[(n - i) % C::kKeySlots], (n - i) / C::kKeySlots & 1);
    for (int i = 0; i < C::kConv; ++i, ++n)  // an end for each group that converts
      if (wait(&kempty[n % C::kKeySlots], n / C::kKeySlots ^ 1) && lane == 0) {
        s_unit[n % C::kKeySlots].tile1 = s_unit[n % C::kKeySlots].tile0 = 0;
        mbar_arrive(&kfull[n % C::kKeySlots]);
      }
    for (int i = 0; i < C::kRowSlots && m > 0 && landed; ++i) {
      --m;
      landed = mbar_wait_warp(&qfull[m % C::kRowSlots], m / C::kRowSlots & 1);
    }
    if (!landed && lane == 0) report_error(a.err, kErrTimeoutDrain);
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ---------------- products: a warp per tile ----------------
    const int x = warp - kMmaWarp;
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
        if (!C::kReuse || in_b != t.b || in_h != t.kvh || in_tile != tile) {  // as the copies go: another tile of rows
          in_b = t.b, in_h = t.kvh, in_tile = tile;
          if (C::kReuse && m > 0 && leader) umma_commit(&qempty[(m - 1) % C::kRowSlots]);
          if (!wait(&qfull[m % C::kRowSlots], m / C::kRowSlots)) break;
          ++m;
        }
        const uint32_t bd = q_lo + (m - 1) % C::kRowSlots * (C::kRowBytes >> 4), turn = steps & 1;
        const uint32_t idesc = umma_idesc_f16(kTile, (rows_of(t, tile) + 15) & ~15, 0, 0);
        if (!wait(&sempty[x][turn], (steps >> 1) ^ 1)) break;
        tc_fence_after_sync();
        if (leader) {
          const uint32_t d = tmem + (2 * x + turn) * kRows, ak = tmem + C::kColK + (2 * (n & 1) + x) * (D / 2);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) mma_ts(d, ak + 8 * s, bd + (((s >> 2) * C::kBox + (s & 3) * 32) >> 4), idesc, s > 0);
          umma_commit(&sfull[x][turn]);
          if (!C::kReuse) umma_commit(&qempty[(m - 1) % C::kRowSlots]);
        }
      }
      if (leader) umma_commit(&aempty[n & 1]);
    }
    if (ok) {
      if (leader) umma_commit(&done);
      wait(&done, 0);
    }
  } else if (warp >= 8 * kSoft && warp < kLoadWarp) {
    // ---------------- codes to fp16: a thread takes one key's row, a lane of tensor memory ----------------
    const int x = (warp >> 2) & 1, row = tid & (kUnit - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    for (uint32_t n = (warp >> 3) - kSoft; wait(&kfull[n % C::kKeySlots], n / C::kKeySlots); n += C::kConv) {
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
#pragma unroll 2
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
  } else if (warp < 8 * kSoft) {
    // ---------------- weights: a thread takes one key ----------------
    const int x = (warp >> 2) & 1, row = tid & (kUnit - 1), group = warp >> 3;
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
      const uint32_t step0 = steps;
      steps += t.tile1 - t.tile0;
      for (int i = (group - step0) & (kSoft - 1); i < t.tile1 - t.tile0; i += kSoft) {
        const uint32_t step = step0 + i, turn = step & 1, from = tmem + (2 * x + turn) * kRows + lanes;
        const int tile = t.tile0 + i;
        if (C::kReuse) {
          if (in_b != t.b || in_h != t.kvh || in_tile != tile) {
            in_b = t.b, in_h = t.kvh, in_tile = tile;
            if (m > 0 && lane == 0) mbar_arrive(&qempty[(m - 1) % C::kRowSlots]);
            ++m;
          }
        } else {
          m = step + 1;
        }
        const float* z = s_z[(m - 1) % C::kRowSlots];  // there before the scores
        const int rows = rows_of(t, tile), first = t.first + (tile >> a.two) * a.tokens;
        if (!wait(&sfull[x][turn], step >> 1)) break;
        tc_fence_after_sync();
        // In place and each kind of operation for many values at a time, so that none waits for the one before it.  The difference
        // of score and lse comes first, in one operation that rounds nothing but it: log2 e in either before that would round
        // numbers that may be large, and a weight would be off by a factor e^(2^-23 |lse|).
        auto add = [&](float (&v)[32], int col, int lo, int hi, auto careful) {
          constexpr bool kCareful = decltype(careful)::value;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (kCareful && e >= hi) break;
            const float4 z4 = *reinterpret_cast<const float4*>(z + col + e);
            fma2v(v[e], v[e + 1], -a.scale, z4.x, z4.y), mul2(v[e], v[e + 1], -kLog2e);
            fma2v(v[e + 2], v[e + 3], -a.scale, z4.z, z4.w), mul2(v[e + 2], v[e + 3], -kLog2e);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (kCareful && e % 4 == 0 && e >= hi) break;
            v[e] = ex2(v[e]);
            if (kCareful && (e < lo || e >= hi)) v[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (kCareful && e >= hi) break;
            add2(sum[0], sum[1], v[e], v[e + 1]);
            add2(sum[2], sum[3], v[e + 2], v[e + 3]);
          }
        };
        // columns [lo, rows) are rows that see this key
        const int lo = min(max(key0 - first + row, 0), kRows) * a.heads;
        const bool all = key0 - first + (row | 31) <= 0;
#pragma unroll 1
        for (int col = 0; col < rows; col += 32) {
          uint32_t raw[32];
          tmem_ld_32x32b_x32(from + col, raw);
          tmem_ld_wait();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
          if (all && col + 32 <= rows)
            add(v, col, 0, 32, std::false_type());
          else
            add(v, col, lo - col, rows - col, std::true_type());
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sempty[x][turn]);
          if (!C::kReuse) mbar_arrive(&qempty[(m - 1) % C::kRowSlots]);
        }
      }
      float mine = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      if (kSoft == 2) {  // the second group hands its sums to the first
        if (!wait(group ? &oempty[n & 1] : &ofull[n & 1], (n >> 1) ^ group)) break;
        if (group)
          s_other[n & 1][row] = mine;
        else
          mine += s_other[n & 1][row];
        __syncwarp();
        if (lane == 0) mbar_arrive(group ? &ofull[n & 1] : &oempty[n & 1]);
        if (group) continue;
      }
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

template <int D, int kSoft>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& codes, const CUtensorMap& par, const Args& a, int ctas,
                   cudaStream_t s) {
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_weights_i4_kernel<D, kSoft>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, kSoft>::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<D, kSoft>::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_weights_i4_kernel<D, kSoft>, q, codes, par, a);
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
  int tokens = 1, log2 = 0;
  while (2 * tokens * heads <= kRows) tokens *= 2, ++log2;
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
  Args a{T, Hq, Hkv, G, log2, tokens, heads, G > kRows, fast_div(heads), (int)pages, ps / kKvBlock, fast_div(ps / kKvBlock), table, width,
         width * ps, cu, kv_lens, B, scale, lse, weights, begun,
         reinterpret_cast<int*>(begun + ctas), part, dev_err};
  // From a full step of rows per sequence on, weights are most of the work and two groups add them up, below it the conversion does
  // (one group that adds up / two: 32 tokens over 32768 24.7 / 24.0 us, prompts 271 / 192, 64 single tokens 77 / 94).
  if ((long long)T * G >= (long long)kRows * B)
    return D == 128 ? launch<128, 2>(tq, tc, tp, a, ctas, s) : launch<64, 2>(tq, tc, tp, a, ctas, s);
  return D == 128 ? launch<128, 1>(tq, tc, tp, a, ctas, s) : launch<64, 1>(tq, tc, tp, a, ctas, s);
}

}  // namespace wql
