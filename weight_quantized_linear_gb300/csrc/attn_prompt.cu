// attn_prompt.cu -- causal attention over packed prompts, fp16, grouped heads.
//
// For every sequence i (rows cu[i] .. cu[i + 1] - 1 of q, k and v) and head h, row r:
//   o[r] = sum_{j <= r} softmax_j(scale q[r] . k[j]) v[j],  k and v those of head h / (Hq / Hkv)
// One pass over the keys with the running maximum and sum of the softmax in fp32.
//
// A CTA takes two tiles of 128 query rows that read the same keys at a time: the same rows of two heads of a group
// where the group is even, else two consecutive row tiles of one head.  Per key tile of 128, the tensor cores compute
// S = Q K^T into tensor memory (tcgen05, both operands in shared memory), the tile's four softmax warps turn it
// into weights P -- thread r owns row r, so neither maximum nor sum needs an exchange -- and write them over S as
// fp16, and the tensor cores add P V to the tile's accumulator, P from tensor memory.  While one tile's softmax runs,
// the tensor cores work on the other's products.  K and V tiles arrive by TMA in a ring of kSlots 128-row tiles.
//
// What bounds it: with heads of 128, 2 x (S 128 + O 128) columns fill tensor memory, so a tile's next S waits for its P
// to be used, and a tile's step takes its softmax (1000 cycles), its turn at the tensor cores and its two products (at least
// 512 cycles each; the queue takes P V in 400 and Q K^T, which reads shared memory at its full bandwidth, in 650): 3000
// cycles for the 2048 that the two tiles' products take by themselves.  With heads of 64, P has columns of its own and S does
// not wait for it; then the two softmaxes, which run at the same time, take 2300 cycles a step.
//
// The softmax's latency is why a step's weights are computed with the maximum as it was, without looking for the new
// one: as long as they add up to less than 2^15, none of them is too large for fp16, and the sum is needed anyway.
// Only a step with more looks for its maximum, rescales the accumulator and computes its weights again (with the
// maximum found in every step, and its growth by 2^8 as the sign to rescale, 16384 tokens of 32 heads take 1.44 ms
// instead of 1.38 to 1.41, in bursts of 20 to 50 calls; over seconds, with the card at its power limit, 1.46 to 1.50).  The
// softmax warps rescale the accumulator themselves, when the product that was added to it last is complete: S(j) complete
// implies that where P is written over S, since P V(j - 1) was queued before it.
//
// One CTA per SM walks through the pairs of tiles, those with the most keys first and every second round in the
// opposite order, which evens out what the CTAs get.  One warp finds the next pair while the current one is worked on,
// and loads and products of the next begin before the outputs of this one are written: a CTA per pair spent about
// 8 us per pair outside the loop over its keys (nine packed prompts of 412 to 3700 tokens, 32 heads: 404 us instead of
// 371).
//
// The weights are rounded to fp16, which the product with fp16 values asks for; their sums are not.  That is off by 2.3e-4 to
// 2.7e-4 of the output's norm, of which 2.0e-4 is the output's own rounding.  A second product with what the rounding leaves
// would make three of a tile's two products per step, half as much tensor work again (16384 tokens: a floor of 1.72 ms instead
// of 1.15): not taken.
//
// Rows see nothing behind them: scores above the diagonal are replaced, not added to.  V rows behind a row would meet
// its zero weights in the product, so in the tiles on the diagonal one warp first replaces V values that are not
// finite by zero and notes the first such key of each channel; rows from that key on get NaN there at the end.
#include <atomic>
#include <climits>

#include "attn.cuh"
#include "internal.h"

namespace wql {
namespace {

constexpr int kTile = 128;                  // query rows and keys of a tile
// warps 0-3, 4-7: softmax of tiles 0, 1; 8: TMA; 9, 10: products of tiles 0, 1; 11: V check; 12: next pair; 13-15: none
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCheckWarp = 11, kNextWarp = 12;
constexpr int kSorted = 128;                // up to so many sequences, the pairs are sorted by their keys
constexpr float kTop = 7.0f;                // the largest weight after a rescale is 2^7, the 128 of a step at most 2^14
constexpr float kMost = 32768.f;            // and a step whose weights come to more than 2^15 asks for the next
// Scores are scaled and the maximum subtracted in one instruction, which does not round the product, while the maximum is a
// rounded number: they differ by up to 2^-24 of it, a factor that all the weights of a row share.  Where it may count, every
// step looks for the maximum and rounds the products first, as the maximum was.
constexpr float kLarge = 1048576.f;
// The maximum of keys whose scores are all minus infinity.  Their weights are zero by it, and the first finite score that
// follows has an infinite one, which makes its step ask for the maximum.
constexpr float kNoMax = -3e38f;
// registers per thread: launched with 128; the softmax warpgroups take 208, the others give down to 48
// (256 x 208 + 256 x 48 = 65536 = 512 x 128)
constexpr int kSoftmaxRegs = 208, kOtherRegs = 48;

template <int D>
struct Cfg {
  static constexpr int kBox = kTile * 128;            // 128 rows of 64 fp16, 128-byte swizzle
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;    // a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 8;
  // D = 64 leaves room in tensor memory for P beside S, so that the next S is computed while this one's softmax runs.  The
  // products are then half of the softmax's work at most, and the tiles need not take turns.
  static constexpr bool kBeside = D == 64;
  static constexpr int kColO = 2 * kTile, kColP = kBeside ? kColO + 2 * D : 0;  // tensor memory columns; S from 0
  static constexpr int kStrideP = kBeside ? kTile / 2 : kTile;                    // between the tiles' P
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kSmem = kOffRing + kSlots * kTileBytes + 1024;  // and alignment of the start
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

// Start and length of sequence b; an invalid one has no rows.
__device__ __forceinline__ int2 sequence(const Args& a, int b) {
  const int s = a.cu[b], e = a.cu[b + 1];
  if (s < 0 || e < s || e > a.T) {
    report_error(a.err, kErrBadIndex);
    return make_int2(0, 0);
  }
  return make_int2(s, e - s);
}

// Slot and phase of a ring.
template <int N>
struct Ring {
  int slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// A pair of tiles: rows r0 .. + 127 of head h0 and r1 .. + 127 of head h1 of a sequence, with n0 and n1 key tiles (n1 = 0:
// there is no second one).  V tiles from jcheck on lie on a diagonal.
struct Pair {
  int start, len, r0, r1, h0, h1, n0, n1, nmax, jcheck;
  __device__ __forceinline__ Pair(const Args& a, const int4& v) {  // {start, length (-1: no more pairs), first row, head}
    start = v.x, len = v.y, r0 = v.z;
    h0 = a.pair ? 2 * v.w : v.w, h1 = a.pair ? h0 + 1 : h0;
    r1 = a.pair ? r0 : r0 + kTile;
    n0 = r0 / kTile + 1, n1 = r1 < len ? r1 / kTile + 1 : 0;
    nmax = max(n0, n1);
    jcheck = (n1 > 0 ? min(n0, n1) : n0) - 1;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const Args a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  // [parity of the pair]: first key (in the sequence) whose V value of this channel is not finite, and whether any is
  __shared__ int bad[2][D], any_bad[2];
  __shared__ int4 s_pair[2];
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t qbar, qfree;             // Q tiles landed; not read any more
  __shared__ uint64_t full[C::kSlots], empty[C::kSlots];
  __shared__ uint64_t sbar[2], pbar[2];        // [tile] S complete; P written (4 warps)
  __shared__ uint64_t obar[2], ofree[2];       // [tile] O complete; O read (4 warps)
  __shared__ uint64_t sfree[2], pfree[2];      // [tile] P beside S: S read (4 warps); P used
  __shared__ uint64_t vbar[2][2], cbar[2][2];  // [parity of the pair][first, second V tile on a diagonal] landed; checked
  __shared__ uint64_t pair_full[2], pair_empty[2];
  __shared__ uint64_t turn[2];                 // [tile] its products may be queued
  __shared__ uint64_t done;                    // every product (both tiles)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    mbar_init(&qbar, 1), mbar_init(&qfree, 2), mbar_init(&done, 2);
    for (int s = 0; s < C::kSlots; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&turn[x], 1), mbar_init(&sbar[x], 1), mbar_init(&pbar[x], 4), mbar_init(&obar[x], 1), mbar_init(&ofree[x], 4);
      mbar_init(&sfree[x], 4), mbar_init(&pfree[x], 1);
      for (int k = 0; k < 2; ++k) mbar_init(&vbar[x][k], 1), mbar_init(&cbar[x][k], 1);
      mbar_init(&pair_full[x], 1), mbar_init(&pair_empty[x], 4 + 8);  // TMA, product, check and softmax warps
      any_bad[x] = 0;
    }
    fence_mbarrier_init();
    mbar_arrive(&turn[0]);
  }
  for (int i = tid; i < 2 * D; i += kThreads) bad[i / D][i % D] = INT_MAX;
  if (warp == kMmaWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  grid_dependency_wait();  // everything before this line overlaps the end of the preceding kernel
  grid_dependents_launch();

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp && lane == 0) {
      // ---------------- Q, then K(0), V(0), K(1), V(1) .. into the ring ----------------
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      Ring<C::kSlots> ring;
      int issued = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_bounded(bar, phase & 1)) {
          report_error(a.err, kErrTimeoutEmpty);
          ok = false;
        }
        return ok;
      };
      auto load_q = [&](int x, int h, int row) {
        for (int b = 0; b < C::kBoxes; ++b) tma_load_3d(smem + x * C::kTileBytes + b * C::kBox, &tm_q, &qbar, 64 * b, h, row);
      };
      for (int it = 0; wait(&pair_full[it & 1], it >> 1); ++it) {
        const int4 v = s_pair[it & 1];
        mbar_arrive(&pair_empty[it & 1]);
        if (v.y < 0) break;
        const Pair p(a, v);
        const int kvh = p.h0 / a.G;
        if (!wait(&qfree, (it & 1) ^ 1)) break;
        mbar_arrive_expect_tx(&qbar, (p.n1 > 0 ? 2 : 1) * C::kTileBytes);
        load_q(0, p.h0, p.start + p.r0);
        for (int i = 0; i < 2 * p.nmax && wait(&empty[ring.slot], ring.phase ^ 1); ++i) {
          uint8_t* dst = smem + C::kOffRing + ring.slot * C::kTileBytes;
          mbar_arrive_expect_tx(&full[ring.slot], C::kTileBytes);
          for (int b = 0; b < C::kBoxes; ++b)
            tma_load_3d(dst + b * C::kBox, i & 1 ? &tm_v : &tm_k, &full[ring.slot], 64 * b, kvh, p.start + (i >> 1) * kTile);
          if (i == 0 && p.n1 > 0) load_q(1, p.h1, p.start + p.r1);  // the second Q tile behind the first K tile
          ring.next();
          ++issued;
        }
      }
      // copies that may still be in flight land before the kernel ends
      for (int i = 0; i < C::kSlots && i < issued; ++i) {
        if (ring.slot == 0) ring.phase ^= 1;
        ring.slot = ring.slot == 0 ? C::kSlots - 1 : ring.slot - 1;
        if (!mbar_wait_bounded(&full[ring.slot], ring.phase)) {
          report_error(a.err, kErrTimeoutDrain);
          break;
        }
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ---------------- the tensor cores' work: a warp per tile ----------------
      // Products are queued only a few deep, so what one warp spent on waits and commits between them was time in which
      // the tensor cores had nothing to do (one warp for both tiles: 1.69 instead of 1.45 ms for 16384 tokens, 32
      // heads).  Each warp waits for what its next products need while the other's are queued, and they take turns in
      // queueing them: left to themselves, the two tiles fall into step, and both softmaxes run while the tensor cores
      // wait (1.73 ms).  A whole warp walks through this, so that what the instructions take is uniform and stays in
      // uniform registers; under a branch on the lane every operand of every product would be moved there first.
      const int x = warp - kMmaWarp;
      const bool leader = elect_one();
      const uint32_t idesc_s = umma_idesc_f16(kTile, kTile, 0, 0) | a.negate;
      constexpr uint32_t idesc_o = umma_idesc_f16(kTile, D, /*A from TMEM*/ 0, /*B MN-major*/ 1);
      const uint32_t ring_lo = smem_u32(smem + C::kOffRing) >> 4;
      const uint32_t q_desc = (1u << 16) + ((smem_u32(smem) + x * C::kTileBytes) >> 4);
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
      auto qk = [&](int slot) {  // S = Q K^T, K in `slot`
        const uint32_t bd = (1u << 16) + ring_lo + slot * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = ((s >> 2) * C::kBox + (s & 3) * 32) >> 4;
            mma_ss(ts, q_desc + off, bd + off, idesc_s, s > 0);
          }
          umma_commit(&sbar[x]);
        }
      };
      auto pv = [&](int slot, uint32_t acc) {  // O (+)= P V, V in `slot`
        const uint32_t bd = ((uint32_t)(C::kBox >> 4) << 16) + ring_lo + slot * (C::kTileBytes >> 4);
        if (leader) {
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s) mma_ts(to, tp + s * 8, bd + ((s * 2048) >> 4), idesc_o, s > 0 ? 1u : acc);
        }
      };
      Ring<C::kSlots> rk, rv;                 // K(j + 1), V(j)
      int pcount = 0, ocount = 0, turns = 0;  // phases of pbar, of obar / ofree, and of turn
      int scount = 0;                         // S so far
      auto my_turn = [&]() { return C::kBeside || wait(&turn[x], turns++); };
      auto pass = [&]() {
        if (!C::kBeside && leader) mbar_arrive(&turn[x ^ 1]);
      };
      auto s_free = [&]() {  // S may be written: its softmax has read it, where P does not say so
        const bool r = !C::kBeside || scount == 0 || wait(&sfree[x], scount - 1);
        ++scount;
        return r;
      };
      for (int it = 0; wait(&pair_full[it & 1], it >> 1); ++it) {
        const int4 v = s_pair[it & 1];
        __syncwarp();
        if (leader) mbar_arrive(&pair_empty[it & 1]);
        if (v.y < 0) break;
        const Pair p(a, v);
        const int n = x ? p.n1 : p.n0;
        const bool signals = x == (p.n1 > 0);  // this warp tells the check warp about V tiles
        // S of the first key tile; the S columns are free, since the products that read their last P come before.  A
        // tile that does not exist, or has fewer keys, follows the ring all the same.
        if (!wait(&qbar, it) || !wait(&full[rk.slot], rk.phase) || !my_turn()) break;
        if (n > 0 && !s_free()) break;
        tc_fence_after_sync();
        if (n > 0) qk(rk.slot);
        pass();
        release(&empty[rk.slot], n > 0);
        if (n <= 1) release(&qfree, n > 0);
        rv = rk;
        rv.next();
        rk = rv;
        rk.next();
        if (signals) {
          if (p.jcheck == 0 && wait(&full[rv.slot], rv.phase) && leader) mbar_arrive(&vbar[it & 1][0]);
          if (p.nmax - 1 == p.jcheck && leader) mbar_arrive(&vbar[it & 1][1]);  // there is no second one
        }
        for (int j = 0; j < p.nmax && wait(&full[rv.slot], rv.phase); ++j) {
          if (j + 1 < p.nmax && !wait(&full[rk.slot], rk.phase)) break;
          if (C::kBeside && j + 1 < n) {
            if (!s_free()) break;
            tc_fence_after_sync();
            qk(rk.slot);
          }
          if (j < n) {
            if (!wait(&pbar[x], pcount++)) break;
            // the accumulator is taken over when the softmax warps have read that of the pair before
            if (j == 0 && ocount > 0 && !wait(&ofree[x], ocount - 1)) break;
            if (j >= p.jcheck && !wait(&cbar[it & 1][j - p.jcheck], it >> 1)) break;
          }
          if (!my_turn()) break;
          tc_fence_after_sync();
          if (j < n) {
            pv(rv.slot, j > 0);
            if (C::kBeside) release(&pfree[x], true);
            if (j + 1 == n) {
              release(&obar[x], true);
              ++ocount;
            }
          }
          if (!C::kBeside && j + 1 < n) qk(rk.slot);
          pass();
          if (j + 1 < p.nmax) {
            release(&empty[rv.slot], j < n);
            release(&empty[rk.slot], j + 1 < n);
            if (j + 2 == n) release(&qfree, true);
            rv = rk;
            rv.next();
            rk = rv;
            rk.next();
            // the next V is checked while its step's softmax runs
            if (signals && j + 1 >= p.jcheck && wait(&full[rv.slot], rv.phase) && leader)
              mbar_arrive(&vbar[it & 1][j + 1 - p.jcheck]);
          } else {
            release(&empty[rv.slot], j < n);  // rk is at K(0) of the next pair
          }
        }
      }
      if (ok) {
        release(&done, true);
        wait(&done, 0);
      }
    } else if (warp == kCheckWarp) {
      // ---------------- V tiles on a diagonal: values that are not finite ----------------
      int base = 0;  // slot of K(0)
      bool ok = true;
      auto wait = [&](uint64_t* bar, int phase) {
        if (ok && !mbar_wait_warp(bar, phase & 1)) {
          if (lane == 0) report_error(a.err, kErrTimeoutFull);
          ok = false;
        }
        return ok;
      };
      for (int it = 0; wait(&pair_full[it & 1], it >> 1); ++it) {
        const int4 v4 = s_pair[it & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&pair_empty[it & 1]);
        if (v4.y < 0) break;
        const Pair p(a, v4);
        int* first_bad = bad[it & 1];
        if (any_bad[it & 1]) {  // of the pair before the last, whose outputs are written
          for (int i = lane; i < D; i += 32) first_bad[i] = INT_MAX;
          __syncwarp();
          if (lane == 0) any_bad[it & 1] = 0;
          __syncwarp();
        }
        for (int k = 0; k < 2; ++k) {
          // not on the ring's own barrier, which goes through phases that this warp does not follow
          if (!wait(&vbar[it & 1][k], it >> 1)) break;
          const int j = p.jcheck + k;
          if (j >= p.nmax) {
            if (lane == 0) mbar_arrive(&cbar[it & 1][k]);
            continue;
          }
          uint4* v = reinterpret_cast<uint4*>(smem + C::kOffRing + (base + 2 * j + 1) % C::kSlots * C::kTileBytes);
          constexpr int kBatch = 4;
          for (int at = lane; at < C::kTileBytes / 16; at += 32 * kBatch) {
            uint4 x[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) x[u] = v[at + 32 * u];
            uint32_t hits = 0;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
              // an exponent of all ones carries into the bit above it
              const uint32_t h = ((x[u].x & 0x7c007c00u) + 0x04000400u) | ((x[u].y & 0x7c007c00u) + 0x04000400u) |
                                 ((x[u].z & 0x7c007c00u) + 0x04000400u) | ((x[u].w & 0x7c007c00u) + 0x04000400u);
              hits |= (h & 0x80008000u) ? 1u << u : 0u;
            }
            for (; hits; hits &= hits - 1) {  // rare
              // chunk c of row r (16-byte units, 8 per 128-byte row) holds channels 8 (c ^ r % 8) of the box
              const int pos = at + 32 * (__ffs(hits) - 1), row = (pos >> 3) & (kTile - 1), box = pos / (kTile * 8);
              const int ch = 64 * box + 8 * ((pos ^ row) & 7), key = j * kTile + row;
              uint16_t* h = reinterpret_cast<uint16_t*>(v + pos);
              for (int e = 0; e < 8; ++e) {
                if ((h[e] & 0x7c00u) != 0x7c00u) continue;
                h[e] = 0;
                if (key < p.len) {
                  atomicMin(&first_bad[ch + e], key);
                  any_bad[it & 1] = 1;
                }
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&cbar[it & 1][k]);
        }
        base = (base + 2 * p.nmax) % C::kSlots;
      }
    } else if (warp == kNextWarp) {
      // ---------------- the pairs of this CTA ----------------
      const int rows_per = a.pair ? kTile : 2 * kTile, nh = a.pair ? a.Hq / 2 : a.Hq;
      auto tiles_of = [&](int len) { return (len + rows_per - 1) / rows_per; };
      constexpr int kPer = kSorted / 32;
      int2 seq[kPer];  // sequences 32 k + lane
      int most = 0, all = 0;
      if (a.B <= kSorted) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          seq[k] = 32 * k + lane < a.B ? sequence(a, 32 * k + lane) : make_int2(0, 0);
          most = max(most, tiles_of(seq[k].y));
          all += tiles_of(seq[k].y);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        all = __reduce_add_sync(0xffffffffu, all);
      }
      auto beyond = [&](int t) {  // row tiles number t and later, of all sequences
        int n = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) n += max(tiles_of(seq[k].y) - t, 0);
        return (int)__reduce_add_sync(0xffffffffu, n);
      };
      int chunk = 0, before = 0;  // more sequences: 32 at a time, with the tiles of those before
      for (int it = 0;; ++it) {
        const long long at = (long long)it * gridDim.x + (it & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        const long long y = at / nh;  // row tile, in order
        int4 out = make_int4(0, -1, 0, (int)(at - y * nh));
        if (a.B <= kSorted) {
          if (y < all) {
            int lo = 0, hi = most;  // beyond(lo) > y >= beyond(hi)
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              (beyond(mid) > (int)y ? lo : hi) = mid;
            }
            int r = (int)y - beyond(lo + 1);  // among the sequences that have a tile lo
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
              const unsigned has = __ballot_sync(0xffffffffu, tiles_of(seq[k].y) > lo);
              const int cnt = __popc(has);
              if (out.y < 0 && r < cnt) {
                const int src = __fns(has, 0, r + 1);
                out.x = __shfl_sync(0xffffffffu, seq[k].x, src);
                out.y = __shfl_sync(0xffffffffu, seq[k].y, src);
                out.z = lo * rows_per;
              }
              r -= cnt;
            }
          }
        } else {
          while (chunk < a.B) {
            const int2 q = chunk + lane < a.B ? sequence(a, chunk + lane) : make_int2(0, 0);
            const int n = tiles_of(q.y);
            int incl = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
              const int o = __shfl_up_sync(0xffffffffu, incl, d);
              if (lane >= d) incl += o;
            }
            const int sum = __shfl_sync(0xffffffffu, incl, 31);
            if (y >= (long long)before + sum) {
              before += sum;
              chunk += 32;
              continue;
            }
            const int src = __ffs(__ballot_sync(0xffffffffu, before + incl > (int)y)) - 1;
            out.x = __shfl_sync(0xffffffffu, q.x, src);
            out.y = __shfl_sync(0xffffffffu, q.y, src);
            out.z = __shfl_sync(0xffffffffu, before + incl - 1, src);  // the longest rows first
            out.z = (out.z - (int)y) * rows_per;
            break;
          }
        }
        if (!mbar_wait_warp(&pair_empty[it & 1], ((it >> 1) & 1) ^ 1)) {
          if (lane == 0) report_error(a.err, kErrTimeoutEmpty);
          break;
        }
        if (lane == 0) {
          s_pair[it & 1] = out;
          mbar_arrive(&pair_full[it & 1]);
        }
        if (out.y < 0) break;
      }
    }
  } else {
    // ---------------- softmax and output of tile x: thread r owns row r ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int x = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * kTile + lanes, to = tmem + C::kColO + x * D + lanes;
    const uint32_t tp = tmem + C::kColP + x * C::kStrideP + lanes;
    const float c = a.scale_log2;
    const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    int scount = 0, ocount = 0, pcount = 0;  // phases of sbar and obar; P so far
    bool ok = true;
    auto wait = [&](uint64_t* bar, int phase) {
      if (ok && !mbar_wait_warp(bar, phase & 1)) {
        if (lane == 0) report_error(a.err, kErrTimeoutMma);
        ok = false;
      }
      return ok;
    };
    for (int it = 0; wait(&pair_full[it & 1], it >> 1); ++it) {
      const int4 v4 = s_pair[it & 1];
      if (v4.y < 0) break;
      const Pair p(a, v4);
      const int n = x ? p.n1 : p.n0;
      float m = 0.f, l0 = 0.f, l1 = 0.f;  // m: what is subtracted from the scaled scores
      for (int j = 0; j < n && wait(&sbar[x], scount++); ++j) {
        tc_fence_after_sync();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, s[i]);
        tmem_ld_wait();
        if constexpr (C::kBeside) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[x]);
        }
        if (j == n - 1) {  // the diagonal tile
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > row) s[i >> 5][i & 31] = 0xff800000u;
        }
        auto row_max = [&]() {  // of the scaled scores, less kTop
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 128; i += 2)
            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1]));
          return __fsub_rn(__fmul_rn(fmaxf(max3(top[0], top[1], top[2]), top[3]), c), kTop);
        };
        if (j == 0) m = fmaxf(row_max(), kNoMax);
        float a0, a1;  // this step's sums
        uint32_t w[C::kBeside ? 4 : 1][16];
        auto weights = [&](float mul) {
          a0 = a1 = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t (&wi)[16] = w[C::kBeside ? i : 0];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float u = __uint_as_float(s[i][2 * e]), v = __uint_as_float(s[i][2 * e + 1]);
              fma2(u, v, mul, -m);
              u = ex2(u), v = ex2(v);
              add2(a0, a1, u, v);
              wi[e] = pack_h2(u, v);
            }
            if constexpr (!C::kBeside) tmem_st_32x32b_x16(tp + 16 * i, wi);
          }
        };
        weights(c);
        if constexpr (C::kBeside) {  // the last P has been used, and O is that of the steps before
          if (pcount > 0 && !wait(&pfree[x], pcount - 1)) break;
          ++pcount;
          tc_fence_after_sync();
        }
        const bool more = a0 + a1 > kMost || fabsf(m) > kLarge;
        if (__any_sync(0xffffffffu, more)) {
          // only the rows that need it, so that a row's roundings do not depend on its neighbours
          const float now = more ? fmaxf(m, row_max()) : m, f = ex2(m - now);
          m = now;
          const bool large = fabsf(m) > kLarge;
          if (__any_sync(0xffffffffu, large)) {
#pragma unroll
            for (int i = 0; i < 128; ++i)
              s[i >> 5][i & 31] = __float_as_uint(__fmul_rn(__uint_as_float(s[i >> 5][i & 31]), large ? c : 1.f));
          }
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
          weights(large ? 1.f : c);
        }
        if constexpr (C::kBeside) {
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_st_32x32b_x16(tp + 16 * i, w[i]);
        }
        l0 += a0, l1 += a1;
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pbar[x]);
      }
      if (n > 0 && wait(&obar[x], ocount++)) {
        tc_fence_after_sync();
        uint32_t o[D / 32][32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) tmem_ld_32x32b_x32(to + 32 * i, o[i]);
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ofree[x]);
        const int r = (x ? p.r1 : p.r0) + row;
        const float inv = 1.f / (l0 + l1);
        if (any_bad[it & 1]) {
#pragma unroll
          for (int i = 0; i < D; ++i)
            if (r >= bad[it & 1][i]) o[i >> 5][i & 31] = 0x7fc00000u;
        }
        if (r < p.len) {
          __half* dst = a.out + ((long long)(p.start + r) * a.Hq + (x ? p.h1 : p.h0)) * D;
#pragma unroll
          for (int i = 0; i < D; i += 16) {
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              h[e] = pack_h2(__uint_as_float(o[i >> 5][(i & 31) + 2 * e]) * inv, __uint_as_float(o[i >> 5][(i & 31) + 2 * e + 1]) * inv);
            st_global_32(dst + i, h, sectors);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&pair_empty[it & 1]);
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
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const Args& a, int ctas, cudaStream_t s) {
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
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<D>, q, k, v, a);
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
  // at most this many pairs: every sequence may end in a ragged tile
  const long long pairs = ((long long)T / (pair ? kTile : 2 * kTile) + (B < T ? B : T)) * (pair ? Hq / 2 : Hq);
  const int ctas = (int)(pairs < num_sms() ? pairs : num_sms());
  return D == 128 ? launch<128>(tq, tk, tv, a, ctas, s) : launch<64>(tq, tk, tv, a, ctas, s);
}

}  // namespace wql
