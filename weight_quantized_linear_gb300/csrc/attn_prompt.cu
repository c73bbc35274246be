// attn_prompt.cu -- causal attention over packed prompts, fp16, grouped heads.
//
// For every sequence i (rows cu[i] .. cu[i + 1] - 1 of q, k and v) and head h, row r:
//   o[r] = sum_{j <= r} softmax_j(scale q[r] . k[j]) v[j],  k and v those of head h / (Hq / Hkv)
// One pass over the keys with the running maximum and sum of the softmax in fp32.
//
// A CTA takes two tiles of 128 query rows that read the same keys: the same rows of two heads of a group where
// the group is even, else two consecutive row tiles of one head.  Per key tile of 128, the tensor cores compute
// S = Q K^T into tensor memory (tcgen05, both operands in shared memory), the tile's four softmax warps turn it
// into weights P -- thread r owns row r, so neither maximum nor sum needs an exchange -- and write them over S as
// fp16, and the tensor cores add P V to the tile's accumulator, P from tensor memory.  While one tile's softmax runs,
// the tensor cores work on the other's products.  2 x (S 128 + O 128) columns fill tensor memory, so a tile's next S
// waits for its P to be used, and a step takes a tile's two products plus its softmax's latency.  K and V tiles
// arrive by TMA in a ring of kSlots 128-row tiles.
//
// That latency is why the weights are computed with the maximum as it was, while the new one is still being found: the
// accumulator is rescaled only when a row's maximum has grown by more than 2^8 since the last time (the weights are
// then still below 2^15), and only then are the step's weights computed again.  The softmax warps rescale it
// themselves: S(j) complete implies P V(j - 1) complete, since both were issued before the commit that signals S(j).
//
// Rows see nothing behind them: scores above the diagonal are replaced, not added to.  V rows behind a row would meet
// its zero weights in the product, so in the tiles on the diagonal two warps first replace V values that are not
// finite by zero and note the first such key of each channel; rows from that key on get NaN there at the end.
#include <atomic>
#include <climits>

#include "internal.h"
#include "tcgen05.cuh"

namespace wql {
namespace {

constexpr int kTile = 128;                  // query rows and keys of a tile
constexpr int kThreads = 384;               // warps 0-3, 4-7: softmax of tiles 0, 1; 8: TMA; 9: MMA; 10, 11: V check
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCheckWarp = 10;
constexpr float kTop = 7.0f;                // the largest weight after a rescale is 2^7 ...
constexpr float kRaise = 8.0f;              // ... and before the next at most 2^15
// registers per thread: launched with 168; the softmax warpgroups take 208, the third gives down to 80
// (2 x 128 x 208 + 128 x 80 = 63488 <= 384 x 168 = 64512)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;

template <int D>
struct Cfg {
  static constexpr int kBox = kTile * 128;            // 128 rows of 64 fp16, 128-byte swizzle
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;    // a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kTileBytes;
  static constexpr int kSmem = kOffBar + 1024 + 1024;  // barriers, and alignment of the start
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct Args {
  const int* cu;
  int B, T, Hq, G, pair;  // pair: the two tiles are heads 2y and 2y + 1; else row tiles 2x and 2x + 1
  float scale_log2;
  uint32_t negate;  // bit of the instruction descriptor that negates Q, for a negative scale
  __half* out;
  unsigned* err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 at once.
__device__ __forceinline__ void fma2(float& x, float& y, float a, float c) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %2};\n mov.b64 r, {%3, %3};\n"
      " fma.rn.f32x2 p, p, q, r;\n mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(c));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%0, %1};\n mov.b64 q, {%2, %3};\n add.rn.f32x2 p, p, q;\n"
      " mov.b64 {%0, %1}, p;\n}"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}" : "=r"(p));
  return p != 0;
}
// Shared-memory descriptors whose upper word (8-row groups 1 KB apart, 128-byte swizzle) is the same for all tiles: the
// lower word is the address / 16 and, for V, the distance of its 64-channel boxes / 16 above it.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "n"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %3};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "n"(kDescHi), "r"(idesc), "r"(acc)
      : "memory");
}

// Start and length of sequence b; an invalid one has no rows.
__device__ __forceinline__ int2 sequence(const Args& a, int b) {
  const int s = a.cu[b], e = a.cu[b + 1];
  if (s < 0 || e < s || e > a.T) {
    report_error(a.err, kErrBadIndex);
    return make_int2(0, 0);
  }
  return make_int2(s, e - s);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Args a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int bad[D];  // first key (in the sequence) whose V value of this channel is not finite
  __shared__ int any_bad;
  __shared__ int s_sum[kThreads / 32];
  __shared__ int3 s_tile;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* qbar = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [1] Q tiles
  uint64_t* full = qbar + 1;                                        // [kSlots]
  uint64_t* empty = full + C::kSlots;                               // [kSlots]
  uint64_t* sbar = empty + C::kSlots;                               // [2] S complete
  uint64_t* pbar = sbar + 2;                                        // [2] P written (4 warps)
  uint64_t* obar = pbar + 2;                                        // [2] O complete
  uint64_t* cbar = obar + 2;                                        // [2] V(jcheck), V(jcheck + 1) checked (2 warps)
  uint64_t* vbar = cbar + 2;                                        // [2] V(jcheck), V(jcheck + 1) landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(vbar + 2);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- the sequence and row tiles of this CTA, counted from the last one: the longest rows start first ----
  const int rows_per = a.pair ? kTile : 2 * kTile;
  const int nh = a.pair ? a.Hq / 2 : a.Hq, tile_index = blockIdx.x / nh, hx = blockIdx.x - tile_index * nh;
  {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += (sequence(a, b).y + rows_per - 1) / rows_per;
    int incl = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      total += s_sum[w];
    }
    const int want = total - 1 - tile_index;
    if (want < 0) return;
    int first = incl - mine;
    if (first <= want && want < incl)
      for (int b = b0; b < b1; ++b) {
        const int2 s = sequence(a, b);
        const int n = (s.y + rows_per - 1) / rows_per;
        if (want < first + n) {
          s_tile = make_int3(s.x, s.y, (want - first) * rows_per);
          break;
        }
        first += n;
      }
  }
  if (tid == 0) {
    any_bad = 0;
    mbar_init(qbar, 1);
    for (int s = 0; s < C::kSlots; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    for (int x = 0; x < 2; ++x) mbar_init(&sbar[x], 1), mbar_init(&pbar[x], 4), mbar_init(&obar[x], 1);
    for (int x = 0; x < 2; ++x) mbar_init(&cbar[x], 2), mbar_init(&vbar[x], 1);
    fence_mbarrier_init();
  }
  for (int i = tid; i < D; i += kThreads) bad[i] = INT_MAX;
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int start = s_tile.x, len = s_tile.y, q0 = s_tile.z;
  // tile x: head h[x], rows r0[x] .. + 127 of the sequence, n[x] key tiles (0: no such tile)
  const int h0 = a.pair ? 2 * hx : hx, h1 = a.pair ? h0 + 1 : h0;
  const int r1 = a.pair ? q0 : q0 + kTile;
  const int n0 = q0 / kTile + 1, n1 = r1 < len ? r1 / kTile + 1 : 0;
  const int nmax = max(n0, n1), kvh = h0 / a.G;
  const int jcheck = (n1 > 0 ? min(n0, n1) : n0) - 1;  // key tiles from here on are on a diagonal

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp && lane == 0) {
      // ---------------- Q, then K(0), V(0), K(1), V(1) .. into the ring ----------------
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      mbar_arrive_expect_tx(qbar, (n1 > 0 ? 2 : 1) * C::kTileBytes);
      for (int b = 0; b < C::kBoxes; ++b) tma_load_3d(smem + b * C::kBox, &tm_q, qbar, 64 * b, h0, start + q0);
      int issued = 0;
      bool ok = true;
      for (int i = 0; i < 2 * nmax && ok; ++i) {
        const int slot = i % C::kSlots;
        if (!mbar_wait_bounded(&empty[slot], ((i / C::kSlots) & 1) ^ 1)) {
          report_error(a.err, kErrTimeoutEmpty);
          ok = false;
          break;
        }
        uint8_t* dst = smem + C::kOffRing + slot * C::kTileBytes;
        mbar_arrive_expect_tx(&full[slot], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
          tma_load_3d(dst + b * C::kBox, i & 1 ? &tm_v : &tm_k, &full[slot], 64 * b, kvh, start + (i >> 1) * kTile);
        if (i == 0 && n1 > 0)  // the second Q tile behind the first K tile
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(smem + C::kTileBytes + b * C::kBox, &tm_q, qbar, 64 * b, h1, start + r1);
        ++issued;
      }
      // copies that may still be in flight land before the kernel ends
      if (!mbar_wait_bounded(qbar, 0)) report_error(a.err, kErrTimeoutDrain);
      for (int i = max(0, issued - C::kSlots); i < issued; ++i)
        if (!mbar_wait_bounded(&full[i % C::kSlots], (i / C::kSlots) & 1)) {
          report_error(a.err, kErrTimeoutDrain);
          break;
        }
    } else if (warp == kMmaWarp) {
      // ---------------- the tensor cores' work, issued by one thread ----------------
      // The whole warp walks through this, so that what the instructions take is uniform and stays in uniform
      // registers; under a branch on the lane every operand of every product would be moved there first (16384 tokens,
      // 32 heads: 1.82 ms).
      const bool leader = elect_one();
      const uint32_t idesc_s = umma_idesc_f16(kTile, kTile, 0, 0) | a.negate;
      constexpr uint32_t idesc_o = umma_idesc_f16(kTile, D, /*A from TMEM*/ 0, /*B MN-major*/ 1);
      const uint32_t q_lo = smem_u32(smem) >> 4, ring_lo = smem_u32(smem + C::kOffRing) >> 4;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_warp(bar, phase & 1)) {
          if (leader) report_error(a.err, kErrTimeoutMma);
          ok = false;
        }
        return ok;
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
      };
      auto qk = [&](int x, int slot) {  // S_x = Q_x K^T, K in `slot`
        const uint32_t ad = (1u << 16) + q_lo + x * (C::kTileBytes >> 4), bd = (1u << 16) + ring_lo + slot * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = ((s >> 2) * C::kBox + (s & 3) * 32) >> 4;
            mma_ss(tmem + x * kTile, ad + off, bd + off, idesc_s, s > 0);
          }
        }
      };
      auto pv = [&](int x, int slot, uint32_t acc) {  // O_x (+)= P_x V, V in `slot`
        const uint32_t bd = ((uint32_t)(C::kBox >> 4) << 16) + ring_lo + slot * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s)
            mma_ts(tmem + 2 * kTile + x * D, tmem + x * kTile + s * 8, bd + ((s * 2048) >> 4), idesc_o, s > 0 ? 1u : acc);
        }
      };
      wait(qbar, 0);
      wait(&full[0], 0);
      if (ok) {
        tc_fence_after_sync();
        qk(0, 0);
        commit(&sbar[0]);
        if (n1 > 0) {
          qk(1, 0);
          commit(&sbar[1]);
        }
        if (C::kSlots < 2 * nmax) commit(&empty[0]);
      }
      if (jcheck == 0 && wait(&full[1], 0) && leader) mbar_arrive(&vbar[0]);
      int sv = 1, pv_phase = 0, sk = 2, k_phase = 0;  // slots and phases of V(j) and K(j + 1)
      for (int j = 0; j < nmax && ok; ++j) {
        const int iv = 2 * j + 1, ik = 2 * j + 2;  // ring items V(j) and K(j + 1)
        wait(&full[sv], pv_phase);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int n = x ? n1 : n0;
          if (j >= n || !wait(&pbar[x], j)) continue;
          if (j >= jcheck && !wait(&cbar[j - jcheck], 0)) continue;
          tc_fence_after_sync();
          pv(x, sv, j > 0);
          if (j + 1 < n && wait(&full[sk], k_phase)) {
            tc_fence_after_sync();
            qk(x, sk);
            commit(&sbar[x]);
          } else if (ok) {
            commit(&obar[x]);
          }
        }
        if (ok && iv + C::kSlots < 2 * nmax) commit(&empty[sv]);
        if (ok && ik + C::kSlots < 2 * nmax) commit(&empty[sk]);
        sv += 2;
        if (sv >= C::kSlots) sv -= C::kSlots, pv_phase ^= 1;
        sk += 2;
        if (sk >= C::kSlots) sk -= C::kSlots, k_phase ^= 1;
        // the next V is checked while its step's softmax runs
        if (j + 1 >= jcheck && j + 1 < nmax && wait(&full[sv], pv_phase) && leader) mbar_arrive(&vbar[j + 1 - jcheck]);
      }
    } else if (warp >= kCheckWarp) {
      // ---------------- V tiles on a diagonal: values that are not finite ----------------
      for (int j = jcheck; j < nmax; ++j) {
        const int i = 2 * j + 1;
        // not on the ring's own barrier, which goes through phases that these warps do not follow
        if (!mbar_wait_warp(&vbar[j - jcheck], 0)) {
          if (lane == 0) report_error(a.err, kErrTimeoutFull);
          break;
        }
        uint4* v = reinterpret_cast<uint4*>(smem + C::kOffRing + (i % C::kSlots) * C::kTileBytes);
        constexpr int kBatch = 4;
        for (int at = tid - kCheckWarp * 32; at < C::kTileBytes / 16; at += 64 * kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) x[u] = v[at + 64 * u];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e)  // an exponent of all ones survives the carry into the bit above it
              hit |= (((w[e] & 0x7c007c00u) + 0x04000400u) & 0x80008000u) != 0;
            if (!hit) continue;
            // chunk c of row r (16-byte units, 8 per 128-byte row) holds channels 8 (c ^ r % 8) of the box
            const int p = at + 64 * u, row = (p >> 3) & (kTile - 1), box = p / (kTile * 8);
            const int ch = 64 * box + 8 * ((p ^ row) & 7), key = j * kTile + row;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t m = 0x7c00u << (16 * (e & 1));
              if ((w[e >> 1] & m) != m) continue;
              w[e >> 1] &= ~(0xffffu << (16 * (e & 1)));
              if (key < len) {
                atomicMin(&bad[ch + e], key);
                any_bad = 1;
              }
            }
            v[p] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cbar[j - jcheck]);
      }
    }
  } else {
    // ---------------- softmax and output of tile x: thread r owns row r ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2, n = x ? n1 : n0, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * kTile + lanes, to = tmem + 2 * kTile + x * D + lanes;
    const float c = a.scale_log2;
    float m = 0.f, l0 = 0.f, l1 = 0.f;  // m: what is subtracted from the scaled scores
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp(&sbar[x], j & 1)) {
        if (lane == 0) report_error(a.err, kErrTimeoutMma);
        ok = false;
        break;
      }
      tc_fence_after_sync();
      uint32_t s[4][32];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, s[i]);
      tmem_ld_wait();
      if (j == n - 1) {  // the diagonal tile
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i > row) s[i >> 5][i & 31] = 0xff800000u;
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 128; i += 2)
        top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1]));
      const float up = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c - kTop;
      if (j == 0) m = up;
      float a0, a1;  // this step's sums
      auto weights = [&]() {
        a0 = a1 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float u = __uint_as_float(s[i][2 * e]), v = __uint_as_float(s[i][2 * e + 1]);
            fma2(u, v, c, -m);
            u = ex2(u), v = ex2(v);
            add2(a0, a1, u, v);
            p[e] = pack_h2(u, v);
          }
          tmem_st_32x32b_x16(ts + 16 * i, p);
        }
      };
      weights();
      if (__any_sync(0xffffffffu, up > m + kRaise)) {
        const float now = fmaxf(m, up), f = ex2(m - now);
        m = now;
        l0 *= f, l1 *= f;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + i, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
          tmem_st_32x32b_x32(to + i, o);
        }
        weights();
      }
      l0 += a0, l1 += a1;
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&pbar[x]);
    }
    if (n > 0 && ok) {
      if (!mbar_wait_warp(&obar[x], 0)) {
        if (lane == 0) report_error(a.err, kErrTimeoutMma);
      } else {
        mbar_wait_warp(&cbar[nmax - 1 - jcheck], 0);  // complete already where this tile used it
        tc_fence_after_sync();
        const int r = (x ? r1 : q0) + row;
        const float inv = 1.f / (l0 + l1);
        const bool poison = any_bad != 0;
        // through the tile's Q rows, which are not needed any more, so that whole lines are written
        constexpr int kChunks = D / 8;  // 16-byte chunks of a row
        uint4* stage = reinterpret_cast<uint4*>(smem + x * C::kTileBytes) + (warp & 3) * 32 * kChunks;
#pragma unroll
        for (int i = 0; i < D; i += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + i, o);
          tmem_ld_wait();
          if (poison) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (r >= bad[i + e]) o[e] = 0x7fc00000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              h[k] = pack_h2(__uint_as_float(o[e + 2 * k]) * inv, __uint_as_float(o[e + 2 * k + 1]) * inv);
            stage[lane * kChunks + (((i + e) >> 3) ^ (lane & (kChunks - 1)))] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        __syncwarp();
        const int rw = (x ? r1 : q0) + (warp & 3) * 32;  // the warp's first row
        __half* dst = a.out + ((long long)(start + rw) * a.Hq + (x ? h1 : h0)) * D;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int at = i * 32 + lane, rr = at / kChunks, ch = at % kChunks;
          if (rw + rr < len)
            *reinterpret_cast<uint4*>(dst + (long long)rr * a.Hq * D + 8 * ch) = stage[rr * kChunks + (ch ^ (rr & (kChunks - 1)))];
        }
      }
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

bool tensor_map(CUtensorMap* m, const uint16_t* p, int D, int heads, int T, long long stride, std::string* err) {
  return make_tmap_3d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p, D, heads, T, (uint64_t)D * 2, (uint64_t)stride * 2, 64, 1, kTile,
                      CU_TENSOR_MAP_SWIZZLE_128B, err);
}

template <int D>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Args& a, dim3 grid, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  attn_prompt_kernel<D><<<grid, kThreads, C::kSmem, s>>>(q, k, v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prompt(const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                               const uint16_t* v, long long v_stride, int T, int Hq, int Hkv, int D, const int* cu, int B,
                               float scale, uint16_t* out, unsigned* dev_err, cudaStream_t s, std::string* err) {
  CUtensorMap tq, tk, tv;
  if (!tensor_map(&tq, q, D, Hq, T, q_stride, err) || !tensor_map(&tk, k, D, Hkv, T, k_stride, err) ||
      !tensor_map(&tv, v, D, Hkv, T, v_stride, err))
    return cudaErrorInvalidValue;
  const int G = Hq / Hkv, pair = G % 2 == 0;
  // a scale of zero keeps a trace of itself, so that masked scores stay minus infinity
  const float mag = scale < 0.f ? -scale : scale;
  Args a{cu, B, T, Hq, G, pair, (mag < 1e-30f ? 1e-30f : mag) * 1.4426950408889634f, scale < 0.f ? 1u << 13 : 0u,
         reinterpret_cast<__half*>(out), dev_err};
  // every sequence may end in a ragged tile
  const int rows_per = pair ? kTile : 2 * kTile;
  const long long tiles = (long long)T / rows_per + (B < T ? B : T);
  const long long ctas = tiles * (pair ? Hq / 2 : Hq);
  if (ctas > INT_MAX) {
    *err = "too many row tiles and heads";
    return cudaErrorInvalidConfiguration;
  }
  const dim3 grid((unsigned)ctas);
  return D == 128 ? launch<128>(tq, tk, tv, a, grid, s) : launch<64>(tq, tk, tv, a, grid, s);
}

}  // namespace wql
