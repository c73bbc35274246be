// kv_weights_i4.cu -- the attention weight that every cached token gets from packed chunks of rows, added to running sums:
//   weights[b, kvh, t] += sum over the rows r of sequence b that see t, and the query heads h of kvh's group, of
//                         exp(scale q[r, h] . k[t] - lse[r, h]),   k = code * s + lo, rounded to fp16.
//
// The sums run over rows, so a warp keeps 32 keys as the first operand of its products (mma.sync, 16 keys x 8 rows x 16
// channels) in registers, made fp16 there: a lane of the fragment needs two keys' rows, and as the products do not mind the
// order of the channels, it takes D / 8 contiguous bytes of codes of each, and the same channels of the rows of q.  K is read
// from memory once.  A lane holds two keys' scores of two rows at a time, turns them into weights and adds them up.
//
// A unit is 384 keys of a K/V head, a step a tile of up to 64 rows (token, query head) of a unit.  One warp of a CTA finds the
// units, looks up their pages and has TMA bring codes and tiles of q into two rings; twelve work on 32 keys each, without
// waiting for one another.  The steps of all units are divided evenly over the CTAs, one per SM; sums of units that CTAs share
// go to the workspace, and a second kernel adds them in their order.  What is added to a sum is added by the memory (no load,
// one operation per sum and call, so the order of CTAs does not show).
#include <atomic>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kWarps = 12, kThreads = 32 * (kWarps + 1);
constexpr int kUnit = 32 * kWarps;  // keys of a unit
constexpr int kRows = 64;   // rows of a step, where a token has no more heads than that
constexpr int kLead = 1;    // steps that stand for a unit's own cost
constexpr int kKeySlots = 3, kRowSlots = 2;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Cfg {
  static constexpr int kCodes = kUnit * KvI4<D>::kRow;                // K's codes of a unit,
  static constexpr int kKeyBytes = kCodes + kUnit / kKvBlock * 128;   // with the parameters of K and V
};

struct Args {
  int T, Hq, Hkv, G, tokens, rows;  // tokens and rows of a step
  FastDiv by_g;
  int pages, bpp;  // bpp: blocks of a page
  FastDiv by_bpp;
  const int* table;
  int width, cap;
  const int *cu, *kv_lens;
  int B;
  float scale_log2;
  const float* lse;
  float* weights;
  int row_bytes;  // of a tile of q in shared memory
  // the workspace: the unit that each CTA began and left unfinished {sequence, K/V head, unit of it, 1}, whether it went on
  // with one (1) and ended it (2), and the sums of both [CTA][0: of the one found begun, 1: of the one begun][kUnit]
  int4* begun;
  int* went_on;
  float* part;
  unsigned* err;
};

// Steps of the units of a sequence: unit u takes the row tiles from skip(u) on, those before see none of its keys.
struct Shape {
  int units, tiles, per, c;  // per: row tiles that a unit's keys fill as tokens (tokens divides kUnit); c: those before row 0
  __device__ __forceinline__ Shape(const Args& a, const KvChunk& k) {
    units = k.rows > 0 && k.len > 0 ? (k.len - 1) / kUnit + 1 : 0;
    tiles = k.rows > 0 ? (k.rows - 1) / a.tokens + 1 : 0;
    per = kUnit / a.tokens;
    c = k.first >= 0 ? (int)(((unsigned)k.first + a.tokens - 1) / a.tokens) : -(-k.first / a.tokens);
  }
  __device__ __forceinline__ int skip(int u) const { return (int)max((long long)per * u - c, 0LL); }
  __device__ __forceinline__ int cost(int u) const { return kLead + tiles - skip(u); }
  __device__ __forceinline__ long long before(int u) const {  // the cost of units 0 .. u - 1
    const long long u0 = c < 0 ? 0 : min(c / per + 1, u);  // units that skip nothing
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

// D (16 x 8, fp32) = A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
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
  constexpr int kWords = D / 32;  // of codes, per lane and key
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit[kKeySlots];
  __shared__ __align__(8) float s_z[kRowSlots][128];  // -lse of the rows, times log2 e; minus infinity for none
  __shared__ uint64_t kfull[kKeySlots], kempty[kKeySlots], qfull[kRowSlots], qempty[kRowSlots];
  __shared__ long long s_sum[kWarps + 1], s_off;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* q_tiles = smem;
  uint8_t* keys = smem + kRowSlots * a.row_bytes;
  if (tid == 0) {
    for (int i = 0; i < kKeySlots; ++i) mbar_init(&kfull[i], 1), mbar_init(&kempty[i], kWarps);
    for (int i = 0; i < kRowSlots; ++i) mbar_init(&qfull[i], 1), mbar_init(&qempty[i], kWarps);
    fence_mbarrier_init();
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
    __syncthreads();
    long long total = 0;
    for (int w = 0; w <= kWarps; ++w) {
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

  if (warp == kWarps) {
    // ---------------- units, codes, rows ----------------
    if (lane == 0) tma_prefetch_desc(&tm_q), tma_prefetch_desc(&tm_codes), tma_prefetch_desc(&tm_par);
    constexpr int kBlocks = kUnit / kKvBlock;
    // where four blocks lie together, one copy brings them; else each block has a lane and a copy of its own
    const int each = a.bpp % 4 == 0 ? 4 : 1;
    const uint32_t bytes = each * (kKvBlock * L::kRow + 128);
    int4 begun = make_int4(0, 0, 0, 0);
    int went_on = 0;
    uint32_t n = 0, m = 0;  // units, tiles of rows so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      if (ok && !mbar_wait_warp(bar, phase & 1)) {
        if (lane == 0) report_error(a.err, kErrTimeoutEmpty);
        ok = false;
      }
      return ok;
    };
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
          const uint32_t ks = n % kKeySlots;
          const int gb = u * kBlocks + lane * each, blocks = (k.len - 1) / kKvBlock + 1;
          bool there = lane * each < kBlocks && gb < blocks;
          const int pg = (int)quot((uint32_t)gb, a.by_bpp), page = there ? a.table[(long long)b * a.width + pg] : 0;
          if (there && (page < 0 || page >= a.pages)) {
            report_error(a.err, kErrBadIndex);
            there = false;
          }
          if (!wait(&kempty[ks], n / kKeySlots ^ 1)) break;
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
            const uint32_t qs = m % kRowSlots;
            const int t0 = tile * a.tokens;
            // the rows' lse, in registers before the slot is waited for
            float z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 32 * i + lane, tok = (int)quot((uint32_t)row, a.by_g);
              z[i] = tok < a.tokens && t0 + tok < k.rows
                         ? a.lse[(long long)(k.start + t0 + tok) * a.Hq + kvh * a.G + (row - tok * a.G)] * -kLog2e
                         : -INFINITY;  // of no row: no weights
            }
            if (!wait(&qempty[qs], m / kRowSlots ^ 1)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) s_z[qs][32 * i + lane] = z[i];
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_expect_tx(&qfull[qs], a.rows * D * 2);
              for (int i = 0; i < D / 64; ++i)
                tma_load_3d(q_tiles + qs * a.row_bytes + i * (a.row_bytes / (D / 64)), &tm_q, &qfull[qs], 64 * i, kvh * a.G,
                            k.start + t0);
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
    if (wait(&kempty[n % kKeySlots], n / kKeySlots ^ 1) && lane == 0) {
      s_unit[n % kKeySlots].tile1 = s_unit[n % kKeySlots].tile0 = 0;
      mbar_arrive(&kfull[n % kKeySlots]);
    }
    // copies that may still be in flight land before the kernel ends; what was in the slot of the end has been read
    bool landed = true;
    for (int i = 0; i < kKeySlots - 1 && n > 0 && landed; ++i) --n, landed = mbar_wait_warp(&kfull[n % kKeySlots], n / kKeySlots & 1);
    for (int i = 0; i < kRowSlots && m > 0 && landed; ++i) --m, landed = mbar_wait_warp(&qfull[m % kRowSlots], m / kRowSlots & 1);
    if (!landed && lane == 0) report_error(a.err, kErrTimeoutDrain);
    return;
  }

  // ---------------- 32 keys of each unit ----------------
  const int g = lane >> 2, c = lane & 3;
  const bool swap = c >= 2;  // lanes 2 and 3 take their words in another order, so that the loads of q meet no bank twice
  const int half_q = a.row_bytes / (D / 64);  // between the boxes of 64 channels
  // q in the swizzled tile: chunk 4 c + w of 16 bytes, D = 128; 2 c + w, D = 64
  const int box = D == 128 ? (c >> 1) * half_q : 0, chunk0 = D == 128 ? 4 * (c & 1) : 2 * c;
  uint32_t n = 0, m = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    if (ok && !mbar_wait_warp(bar, phase & 1)) {
      if (lane == 0) report_error(a.err, kErrTimeoutFull);
      ok = false;
    }
    return ok;
  };
  int in_b = -1, in_h = -1, in_tile = -1;
  for (; wait(&kfull[n % kKeySlots], n / kKeySlots); ++n) {
    const uint32_t ks = n % kKeySlots;
    const Unit t = s_unit[ks];
    if (t.tile0 == t.tile1) break;
    const int key0 = t.u * kUnit + 32 * warp, in = 16 * (c >> 1) + 8 * (c & 1) + g;  // this lane's key at the end
    // fp16 fragments: step 2 w has the pairs (0, 1) and (2, 3) of word w, step 2 w + 1 (4, 5) and (6, 7)
    uint32_t A[2][2 * kWords][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 32 * warp + 16 * mt + 8 * e + g;
        const uint32_t src = smem_u32(keys + ks * C::kKeyBytes) + row * L::kRow;
        uint32_t w[kWords];
        if constexpr (D == 128) {
          const uint4 v = lds_u128(src + 16 * c);
          w[0] = swap ? v.z : v.x, w[1] = swap ? v.w : v.y, w[2] = swap ? v.x : v.z, w[3] = swap ? v.y : v.w;
        } else {
          const uint2 v = lds_u64(src + 8 * c);
          w[0] = v.x, w[1] = v.y;
        }
        uint32_t p = lds_u32(smem_u32(keys + ks * C::kKeyBytes) + C::kCodes + row / kKvBlock * 128 + row % kKvBlock * 4);
        if (t.u * kUnit + row >= t.len) p = 0u;
        if (!kv_finite(p)) p = 0x7fff7fffu;
        const uint32_t s2 = prmt(p, 0, 0x1010), lo2 = prmt(p, 0, 0x3232);
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          uint32_t h[4];
          kv_values8(w[i], s2, lo2, h);
          if (kv_overflows(p)) {  // rare; of a NaN: no
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = kv_clamp2(h[j]);
          }
          A[mt][2 * i][e] = prmt(h[0], h[1], 0x5410), A[mt][2 * i][2 + e] = prmt(h[2], h[3], 0x5410);
          A[mt][2 * i + 1][e] = prmt(h[0], h[1], 0x7632), A[mt][2 * i + 1][2 + e] = prmt(h[2], h[3], 0x7632);
        }
      }
    fence_proxy_async_smem();  // these reads come before the copies that follow them into the slot
    __syncwarp();
    if (lane == 0) mbar_arrive(&kempty[ks]);
    float sum[2][2][2] = {};  // [keys 16 mt][+ 8 e] of the two rows
    for (int tile = t.tile0; tile < t.tile1; ++tile) {
      if (in_b != t.b || in_h != t.kvh || in_tile != tile) {  // as above: another tile
        in_b = t.b, in_h = t.kvh, in_tile = tile;
        if (m > 0) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&qempty[(m - 1) % kRowSlots]);
        }
        if (!wait(&qfull[m % kRowSlots], m / kRowSlots)) break;
        ++m;
      }
      const uint32_t qs = (m - 1) % kRowSlots, src = smem_u32(q_tiles + qs * a.row_bytes) + box;
      const int t0 = tile * a.tokens, rows = min(t.n - t0, a.tokens) * a.G;
      auto eights = [&](auto careful) {  // some row does not see all of the warp's keys, or is not one of this sequence
        constexpr bool kCareful = decltype(careful)::value;
#pragma unroll 1
        for (int nt = 0; nt < (rows + 7) / 8; ++nt) {
          float d[2][4];
          const int row = 8 * nt + g;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const uint32_t ch = D == 128 ? chunk0 + (w ^ (swap ? 2 : 0)) : chunk0 + w;
            uint4 bq = make_uint4(0u, 0u, 0u, 0u);
            if (!kCareful || row < rows) bq = lds_u128(src + row * 128 + ((ch ^ (row & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              if (w == 0)
                mma_zero(d[mt], A[mt][0], bq.x, bq.y);
              else
                mma_f16_16816(d[mt], A[mt][2 * w], bq.x, bq.y);
              mma_f16_16816(d[mt], A[mt][2 * w + 1], bq.z, bq.w);
            }
          }
          const float2 z = *reinterpret_cast<const float2*>(&s_z[qs][8 * nt + 2 * c]);
          const int r = 8 * nt + 2 * c;
          int tok0 = 0, tok1 = 0;
          if constexpr (kCareful) tok0 = (int)quot((uint32_t)r, a.by_g), tok1 = (int)quot((uint32_t)r + 1, a.by_g);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float p0 = d[mt][2 * e], p1 = d[mt][2 * e + 1];
              fma2v(p0, p1, a.scale_log2, z.x, z.y);
              p0 = ex2(p0), p1 = ex2(p1);
              if constexpr (kCareful) {
                const int last = t.first + t0 - (key0 + 16 * mt + 8 * e + g);
                if (r >= rows || last + tok0 < 0) p0 = 0.f;
                if (r + 1 >= rows || last + tok1 < 0) p1 = 0.f;
              }
              add2(sum[mt][e][0], sum[mt][e][1], p0, p1);
            }
        }
      };
      if (key0 + 31 > t.first + t0 || rows % 8 != 0)
        eights(std::true_type());
      else
        eights(std::false_type());
    }
    // over the four lanes that share a key; lane (g, c) then has key 16 (c >> 1) + 8 (c & 1) + g
    float s[2][2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[mt][e] = sum[mt][e][0] + sum[mt][e][1];
        s[mt][e] += __shfl_xor_sync(0xffffffffu, s[mt][e], 1);
        s[mt][e] += __shfl_xor_sync(0xffffffffu, s[mt][e], 2);
      }
    const float mine = c & 2 ? (c & 1 ? s[1][1] : s[1][0]) : (c & 1 ? s[0][1] : s[0][0]);
    if (t.slot >= 0)
      a.part[((long long)blockIdx.x * 2 + t.slot) * kUnit + 32 * warp + in] = mine;
    else if (key0 + in < t.len)
      atomicAdd(a.weights + ((long long)t.b * a.Hkv + t.kvh) * a.cap + key0 + in, mine);
  }
}

// Adds the sums of the unit that CTA blockIdx.x began and others went on with.
__global__ void __launch_bounds__(kUnit) kv_weights_join_kernel(const Args a, int ctas) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int c = blockIdx.x;
  const int4 it = a.begun[c];
  if (it.w == 0) return;
  const int key = it.z * kUnit + threadIdx.x;
  float sum = a.part[((long long)c * 2 + 1) * kUnit + threadIdx.x];
  for (int i = c + 1; i < ctas; ++i) {
    const int v = a.went_on[i];
    sum += a.part[(long long)i * 2 * kUnit + threadIdx.x];
    if (v != 1) break;
  }
  if (key < min(max(a.kv_lens[it.x], 0), a.cap)) a.weights[((long long)it.x * a.Hkv + it.y) * a.cap + key] += sum;
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& codes, const CUtensorMap& par, const Args& a, int ctas,
                   cudaStream_t s) {
  constexpr int kMost = 2 * (D / 64) * 128 * 128 + kKeySlots * Cfg<D>::kKeyBytes + 1024;  // 128 rows
  static_assert(kMost <= 220 * 1024, "shared memory");
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_weights_i4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kRowSlots * a.row_bytes + kKeySlots * Cfg<D>::kKeyBytes + 1024;
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
  int tokens = 1;  // of a step: a power of two, which divides kUnit
  while (2 * tokens * G <= kRows) tokens *= 2;
  const int rows = tokens * G, tile_rows = (rows + 7) / 8 * 8;
  const uint64_t piece = 128, block = kKvBlock * (D + 8), blocks = (uint64_t)pages * Hkv * (ps / kKvBlock);
  const uint32_t together = ps % 64 == 0 ? 4 : 1;
  CUtensorMap tq, tc, tp;
  if (!make_tmap_3d(&tq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, q, D, Hq, T, (uint64_t)D * 2, (uint64_t)q_stride * 2, 64, G, tokens,
                    CU_TENSOR_MAP_SWIZZLE_128B, err) ||
      !make_tmap_3d(&tc, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, piece, block / piece, blocks, piece, block, piece,
                    kKvBlock * D / 2 / piece, together, CU_TENSOR_MAP_SWIZZLE_NONE, err) ||
      !make_tmap_3d(&tp, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, piece, block / piece, blocks, piece, block, piece, 1, together,
                    CU_TENSOR_MAP_SWIZZLE_NONE, err))
    return cudaErrorInvalidValue;
  float* part = static_cast<float*>(workspace);
  int4* begun = reinterpret_cast<int4*>(part + (size_t)ctas * 2 * kUnit);
  Args a{T, Hq, Hkv, G, tokens, rows, fast_div(G), (int)pages, ps / kKvBlock, fast_div(ps / kKvBlock), table, width,
         width * ps, cu, kv_lens, B, scale * kLog2e, lse, weights, tile_rows * 128 * (D / 64), begun,
         reinterpret_cast<int*>(begun + ctas), part, dev_err};
  return D == 128 ? launch<128>(tq, tc, tp, a, ctas, s) : launch<64>(tq, tc, tp, a, ctas, s);
}

}  // namespace wql
