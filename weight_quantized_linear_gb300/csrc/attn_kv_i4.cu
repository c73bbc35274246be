// attn_kv_i4.cu -- attention of the last Lq tokens of each sequence over the paged 4-bit KV cache, with
// grouped heads: o = softmax(scale q k^T) v, k and v = code * s + lo, keys t <= len - Lq + r for row r.
//
// A unit of work is one (sequence, K/V head, block of 8 NT query rows); the rows of a K/V head are its
// Lq * G (token, query head) pairs, so a K/V head's cache is read once for all the query heads it serves.
// Units are cut into steps of 32 tokens.  The steps of all units, in order, are divided evenly over the
// CTAs (one per SM), whatever the lengths, and a CTA's steps evenly over its warps, each a run of its own.  One
// more warp requests the copies: its lane w keeps warp w's ring of steps filled, across unit boundaries, so that no
// warp waits for another while streaming and a short unit costs no synchronisation.  A warp writes a unit that lies in
// its run; parts of units that span warps are joined in shared memory at the CTA's end.  Parts of units that span CTAs
// go to the workspace; the CTA that finds all the parts of a unit there joins them, in their order, so that no CTA
// waits for another and the result does not depend on who does it.
//
// Mathematics.  Scores: sum_c q_c (code_c s + lo) = s sum_c q_c code_c + lo sum_c q_c, so the matrix product
// runs on the codes.  Masking a nibble in place makes it an fp16 number without any conversion: a code in
// bits 0-3 is the subnormal code * 2^-24 and in bits 4-7 code * 2^-20, exactly; the products of the two
// kinds are kept in two accumulators (or, for V, in different output rows) and scaled apart at the end.
// Values: sum_t p_t (s_t code_t + lo_t) = sum_t (p_t s_t) code_t + sum_t p_t lo_t, with w_t = p_t s_t as the
// fp16 weight of the second matrix product and the last sum in fp32.  The running maximum m is that of
// score + log2 |s|, i.e. of w itself, so the weights use fp16's range however the scales differ between
// tokens; m is raised only when a weight would pass 2^15 (the rescaling is skipped while it is idle).  An s of zero,
// which the format allows, counts as 2^-24 for m.
// What all the codes of a token share is kept out of the sums, which would otherwise grow to hundreds of times the
// result of a long context and carry their truncation and that of the weights with them.  Every second token enters
// the product as 15 - code with the weight -w, so that the accumulators stay small; and with w' the rounded, signed
// weights, 7.5 sum_t w'_t is taken off at the end (one more product, with a matrix of ones, gives that sum where it is
// needed) while p_t (lo_t + 7.5 s_t) goes to the fp32 sum: a weight's rounding then meets code - 7.5.
// A constant row of V has codes 0 and, by the format, s = 1, whatever the size of its value.  Taken as it stands its weight's
// rounding would meet 7.5 instead of 0, and its s would set the maximum that the other tokens' weights are held against.
// So a token with |s| = 1 whose codes are all zero counts as one with s = 2^-24, the least there is: its value stays lo, and
// what its weight's rounding adds vanishes (64 tokens of size 0.05, four of them zero, 16 rows with heads of 128: error
// 4.8e-3 -> 2.6e-4 of the norm, 1.8e-2 -> 3.1e-4 in the worst row).  The codes are looked at only in steps that hold an s of
// 1, on the path that raises the maximum (64 contexts: no change in time, four drafted tokens x 32: 27.9 -> 28.3 us; a vote
// of its own: 61.5 for 59.7).
// Up to four rows leave half of the products' eight columns free: there the same rows stand a second time (kTwin), with
// what the rounding of their weights left as weights.  The output is then off by its own rounding alone
// (2.0e-4 of its norm instead of 2.9e-4).  64 contexts with 4 rows: 59.2 -> 59.9 us; a second set of products instead,
// which more rows would need, 59 -> 67 us, so those keep rounded weights.
//
// mma.sync, not tcgen05: operands come out of registers after the unpacking, 8 rows (the query heads of a K/V
// head) are the narrow side, and a 16-token block with heads of 128 needs 17 products of 16 x 8 x 16 for 8 rows (8 for the
// scores, 8 for the values, one for the weights' sum; 9 with heads of 64), which the SM does in a third of the time in
// which HBM delivers the block.  That holds for decode steps and drafted tokens.  A chunk of a prompt has many more rows, and
// every 16 of them read the cache again: 512 tokens behind 8192 cached ones take 314 us (128 tokens 87, 16 tokens 25; 32
// query and 8 K/V heads of 128); attention_chunks_kv_i4 is for those.
//
// Measured on GB300: 64 ragged contexts up to 8192 tokens, 8 K/V heads of 128 (290 MB) 60 us, of which 47 stream the
// cache at 6.2 TB/s and the rest is finding the range, joining and the launch; one context of 120001 tokens (131 MB) 31 us;
// 16 rows per K/V head with heads of 64 (48 MB) 28 us, half of it the unit's own cost and joins, the rest bound by the
// steps' instructions and their latency (14 us more per 48 MB; issue slots 48 % used by the 12 warps that fit); heads of 64
// with 4 rows, 64 contexts (154 MB) 49 us, one of 120001 tokens (69 MB) 26 us; 700 tokens, 32 K/V heads 7.5 us, bound by its
// chain of latencies.
#include <atomic>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kStep = 32;                       // tokens per step
constexpr int kLead = 3;                        // steps that stand for a unit's own cost
constexpr int kOwnSteps = 48;                   // steps (1536 tokens) up to which a unit may have a CTA of its own
constexpr float kNoMax = -3e38f;                // maximum of nothing, below every score
constexpr float kLeast = 5.9604644775390625e-8f, kLeastLog2 = -24.f;  // the least s above zero, 2^-24
// Weights are kept below 2^15: at each raise of m the largest becomes 2^7, so that those down to 2^-21 of it are normal
// fp16 numbers.
constexpr float kTop = 7.0f, kRaise = 15.0f;

template <int D, int NT>
struct Cfg {
  // as many as registers allow.  More with fewer registers: heads of 64, 8 rows with 19 warps 23.4 us for 23.2 (190 MB:
  // 57 for 59), 16 rows with 15 warps spill and take 37 us for 28.
  static constexpr int kWarps = NT == 1 ? (D == 64 ? 15 : 11) : (D == 64 ? 11 : 7);  // and one: a multiple of 4
  static constexpr int kThreads = 32 * (kWarps + 1);  // and the warp that requests the copies
  static constexpr int kStepBytes = kStep / kKvBlock * KvI4<D>::kBytes;
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kRows = 8 * NT;
  static constexpr int kJoinPitch = D + 4;                                  // floats per row of the join buffer
  static constexpr int kOffJoin = kWarps * kStages * kStepBytes;            // [kWarps][kRows][kJoinPitch] fp32: first parts
  static constexpr int kOffMl = kOffJoin + kWarps * kRows * kJoinPitch * 4; // [first, last part][kWarps][kRows] {m, l}
  static constexpr int kOffFac = kOffMl + 2 * kWarps * kRows * 8;           // [2][kWarps][kRows] {factor, its l, maximum}
  static constexpr int kOffBar = kOffFac + 2 * kWarps * kRows * 16;         // [full, empty][kWarps][kStages] mbarriers
  static_assert(kRows * kJoinPitch * 4 <= kStages * kStepBytes, "a last part takes the warp's ring");
  static constexpr int kSmem = kOffBar + 2 * kWarps * kStages * 8;
};

// (a & b) ^ c in one instruction, b and c in registers.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).  Not volatile, unlike its namesake: the products of a step's
// two blocks may be interleaved.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 h2f2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// A flag with any other value says that the part is not there, so the workspace may hold anything before a call.
constexpr unsigned long long kThere = 0x9d6b2f81c35ae704ull;

// The flags are the only words that CTAs write and read at the same time, by operations that are strong at the GPU's scope.
// The fences around them order the parts before the flags and the flags before the parts that are read; release and acquire
// on top of those cost 0.5 us (64 contexts) to 1.3 us (four drafted tokens x 32).
__device__ __forceinline__ void set_flag(unsigned long long* f, unsigned long long v) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(__cvta_generic_to_global(f)), "l"(v) : "memory");
}
__device__ __forceinline__ bool flag_set(const unsigned long long* f) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(__cvta_generic_to_global(f)) : "memory");
  return v == kThere;
}

struct Args {
  const __half* q;
  long long q_stride;
  int B, Lq, Hq, Hkv, G, RB;  // RB: row blocks per K/V head
  const uint8_t* cache;
  int pages;
  const int* table;
  int width, cap;  // pages of a row of the table, and their tokens
  int split;       // 0: a CTA per unit; 1: the steps of all units evenly over the CTAs
  const int* kv_lens;
  float scale_log2;
  FastDiv bpp, rb;  // blocks per page, row blocks per head
  __half* out;
  float* part;  // [gridDim][2][kRows][D + 4]: O, m, l of the units that end (0) and go on (1) behind the CTA's range
  unsigned long long* flag;  // [gridDim][2]: kThere where that part is complete
  unsigned* err;
};

__device__ __forceinline__ int seq_len(const Args& a, int b) { return min(max(a.kv_lens[b], 0), a.cap); }
// Steps of a unit of sequence b.  Its first kLead steps are no tokens: they stand for what a unit costs beside them (its
// queries, reductions and output), so that the warps that meet many short units get fewer tokens (64 ragged contexts:
// 62 us without, 61, 60 and 59 us with one, two and three lead steps).
__device__ __forceinline__ int seq_steps(const Args& a, int b) {
  const int len = seq_len(a, b);  // may be up to 2^31 - 1
  return len > 0 ? (len - 1) / kStep + 1 + kLead : 0;
}

// Position in the order of all steps: unit (b, hr = head * RB + row block), step s of `n` of that unit.
struct Cursor {
  int b, hr, s, n;
};
__device__ __forceinline__ void advance(const Args& a, Cursor& c, int by) {
  c.s += by;
  while (c.s >= c.n) {
    c.s -= c.n;
    if (++c.hr == a.Hkv * a.RB) {
      c.hr = 0;
      do {
        if (++c.b >= a.B) {
          c.n = INT_MAX;  // past the end: nothing is read there
          return;
        }
        c.n = seq_steps(a, c.b);
      } while (c.n == 0);
    }
  }
}

// Zeros in rows [row0, row0 + count) of a sequence's K/V head, by the whole CTA.
template <int D>
__device__ void zero_rows(const Args& a, int b, int head, int row0, int count) {
  for (int i = threadIdx.x; i < count * (D / 8); i += blockDim.x) {
    const int r = row0 + i / (D / 8);
    if (r < a.Lq * a.G)
      reinterpret_cast<uint4*>(a.out)[(((long long)b * a.Lq + r / a.G) * a.Hq + head * a.G + r % a.G) * (D / 8) + i % (D / 8)] =
          make_uint4(0u, 0u, 0u, 0u);
  }
}

// Whether a token's codes are all zero.
template <int D>
__device__ __forceinline__ bool no_codes(const uint8_t* row) {
  uint32_t any = 0;
#pragma unroll 1
  for (int i = 0; i < KvI4<D>::kRow; i += 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + i);
    any |= x.x | x.y | x.z | x.w;
  }
  return any == 0;
}

template <int D, int NT, bool kTwin>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) attn_kv_i4_kernel(const Args a) {
  static_assert(!kTwin || NT == 1, "rows 0-3 of one tile, twice");
  using C = Cfg<D, NT>;
  using L = KvI4<D>;
  constexpr int kW = C::kWarps, kS = C::kStages;
  constexpr int kKw = D / 32;  // words of K codes per thread and token
  constexpr int kMt = D / 16;  // 16-channel tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::kOffJoin);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  __shared__ int4 s_start[kW];              // the warps' first positions
  __shared__ int4 s_first[kW], s_last[kW];  // {sequence, head and row block, first step of the unit, kPart | kEnds}
  constexpr int kPart = 1, kEnds = 2;       // there is such a part; the unit ends in it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  for (int i = tid; i < 2 * kW * kS; i += C::kThreads) mbar_init(&bars[i], 1);
  fence_mbarrier_init();
  grid_dependency_wait();  // everything before this line overlaps the end of the preceding kernel
  grid_dependents_launch();

  // ---- this CTA's range [n0, n1) of the order of all steps (of its unit's, where each has a CTA) --------
  const int hr_all = a.Hkv * a.RB;
  int n0, n1, quota, incl = 0, mine = 0, b0 = 0, b1 = 0;
  if (!a.split) {
    const int b = (int)blockIdx.x / hr_all;
    if (tid == 0 && a.kv_lens[b] > a.cap) report_error(a.err, kErrBadIndex);
    n0 = kLead, n1 = quota = seq_steps(a, b);  // nothing to even out: no lead steps
    if (n1 == 0) {
      const int head = (int)blockIdx.x % hr_all / a.RB, row0 = (int)blockIdx.x % a.RB * C::kRows;
      zero_rows<D>(a, b, head, row0, C::kRows);
      return;
    }
  } else {  // every warp scans the lengths itself
    const int per = (a.B + 31) / 32;
    b0 = min(lane * per, a.B), b1 = min(b0 + per, a.B);
    for (int b = b0; b < b1; ++b) {
      if (a.kv_lens[b] > a.cap) report_error(a.err, kErrBadIndex);
      mine += seq_steps(a, b) * hr_all;
    }
    incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    // at least one step for every warp of a CTA: a short batch uses fewer CTAs and has fewer parts to join
    quota = max((int)(((unsigned)total + gridDim.x - 1) / gridDim.x), kW);
    n0 = (int)min((unsigned)quota * blockIdx.x, (unsigned)total), n1 = (int)min((unsigned)n0 + quota, (unsigned)total);
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)  // sequences without any token
      if (seq_len(a, b) == 0)
        for (int head = 0; head < a.Hkv; ++head) zero_rows<D>(a, b, head, 0, a.Lq * a.G);
    if (n0 >= n1) return;
  }
  // warp w's run of steps is [run(w), run(w + 1))
  const int quota_w = (n1 - n0 + kW - 1) / kW, warps = (n1 - n0 + quota_w - 1) / quota_w;  // warps with a run
  auto run = [&](int w) { return (int)min((unsigned)n0 + (unsigned)quota_w * w, (unsigned)n1); };
  if (warp < warps) {
    const int at = run(warp);
    if (!a.split) {
      if (lane == 0) s_start[warp] = make_int4((int)blockIdx.x / hr_all, (int)blockIdx.x % hr_all, at, n1);
    } else if (int first = incl - mine; first <= at && at < incl) {
      for (int b = b0; b < b1; ++b) {
        const int n = seq_steps(a, b);
        if (at < first + n * hr_all) {
          s_start[warp] = make_int4(b, (at - first) / n, (at - first) % n, n);
          break;
        }
        first += n * hr_all;
      }
    }
  }
  if (warp < kW && lane == 0) s_first[warp] = s_last[warp] = make_int4(0, 0, 0, 0);
  __syncthreads();

  // ---- the warp that requests: lane w keeps warp w's ring filled ---------------------------------
  if (warp == kW) {
    if (lane < warps) {
      const int bpp = (int)a.bpp.d;
      const uint32_t ring = smem_u32(smem) + lane * kS * C::kStepBytes;
      uint64_t* full = bars + lane * kS;
      uint64_t* empty = bars + (kW + lane) * kS;
      Cursor pc{s_start[lane].x, s_start[lane].y, s_start[lane].z, s_start[lane].w};
      int pn = run(lane);  // next step to request
      const int pn1 = run(lane + 1);
      int slot = 0, pg0 = 0, pg1 = 0, blk = 0, col0 = 0, last = 0;
      uint32_t parity = 1;  // the first round finds every stage free
      auto look_up = [&]() {  // the pages of the two blocks of the step at pc
        blk = (pc.s - kLead) * (kStep / kKvBlock);
        last = (seq_len(a, pc.b) - 1) / kKvBlock;
        col0 = (int)quot(blk, a.bpp);
        const int* row = a.table + (long long)pc.b * a.width;
        pg0 = row[col0];
        pg1 = blk < last ? row[quot(blk + 1, a.bpp)] : pg0;
      };
      auto next = [&](int by) {  // to the next step with tokens
        pn += by;
        if (by && pn < pn1) advance(a, pc, by);
        while (pn < pn1 && pc.s < kLead) {
          pn += 1;
          if (pn < pn1) advance(a, pc, 1);
        }
        if (pn < pn1) look_up();
      };
      next(0);
      unsigned long long since = globaltimer_ns();
      while (pn < pn1) {
        // a test, not a wait: a lane whose stage is in use must not hold up the others
        if (!mbar_test_wait(&empty[slot], parity)) {
          if (globaltimer_ns() - since > kWaitLimitNs) {
            report_error(a.err, kErrTimeoutEmpty);
            break;
          }
          __nanosleep(40);
          continue;
        }
        if ((unsigned)pg0 >= (unsigned)a.pages || (unsigned)pg1 >= (unsigned)a.pages) {
          report_error(a.err, kErrBadIndex);
          if ((unsigned)pg0 >= (unsigned)a.pages) pg0 = 0;
          if ((unsigned)pg1 >= (unsigned)a.pages) pg1 = 0;
        }
        const int head = (int)quot(pc.hr, a.rb), in0 = blk - col0 * bpp, in1 = in0 + 1 < bpp ? in0 + 1 : 0;
        const bool two = blk < last;
        const uint32_t dst = ring + slot * C::kStepBytes;
        const uint8_t* s0 = a.cache + (((long long)pg0 * a.Hkv + head) * bpp + in0) * L::kBytes;
        mbar_arrive_expect_tx(&full[slot], two ? 2 * L::kBytes : L::kBytes);
        if (two && in1 > 0) {
          bulk_load(dst, s0, 2 * L::kBytes, &full[slot]);
        } else {
          bulk_load(dst, s0, L::kBytes, &full[slot]);
          if (two)
            bulk_load(dst + L::kBytes, a.cache + (((long long)pg1 * a.Hkv + head) * bpp + in1) * L::kBytes, L::kBytes,
                      &full[slot]);
        }
        slot = slot + 1 == kS ? 0 : slot + 1;
        parity ^= slot == 0;
        next(1);
        since = globaltimer_ns();
      }
    }
  } else {

    // ---- the units of a warp's run ---------------------------------------------------------------
    const uint8_t* ring = smem + warp * kS * C::kStepBytes;
    uint64_t* full = bars + warp * kS;
    uint64_t* empty = bars + (kW + warp) * kS;
    int slot = 0;
    uint32_t parity = 0;
    bool alive = true;
    const int r0 = run(warp), r1 = run(warp + 1);
    Cursor u{s_start[warp].x, s_start[warp].y, s_start[warp].z, s_start[warp].w};  // of no meaning without a run
    for (int at = r0; at < r1;) {
      const int end = min(at + (u.n - u.s), r1);  // of this warp's part of the unit
      const int len = seq_len(a, u.b), head = (int)quot(u.hr, a.rb), rb = u.hr - head * a.RB;
      const int rows = a.Lq * a.G, row0 = rb * C::kRows;
      // Q fragments: thread (g, c) holds row g's channels of its K words, paired as the codes will be
      uint32_t qf[NT][kKw][4];
      float2 qsum[NT];  // of rows 2c and 2c + 1, scaled
      int lim[NT][2];   // last visible token of those rows
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = row0 + 8 * t + (kTwin ? g & 3 : g);
        float sum = 0.f;
        uint4 raw[kKw];
#pragma unroll
        for (int j = 0; j < kKw; ++j) raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) {
          const int r = row / a.G, hq = head * a.G + row % a.G;
          const __half* src = a.q + ((long long)u.b * a.Lq + r) * a.q_stride + (long long)hq * D + 8 * kKw * c;
#pragma unroll
          for (int j = 0; j < kKw; ++j) raw[j] = __ldg(reinterpret_cast<const uint4*>(src) + j);
        }
#pragma unroll
        for (int j = 0; j < kKw; ++j) {
          // channels 8w + (0,1) (2,3) (4,5) (6,7) -> pairs (0,4) (2,6) of the low nibbles, (1,5) (3,7) of the high
          qf[t][j][0] = prmt(raw[j].x, raw[j].z, 0x5410u);
          qf[t][j][1] = prmt(raw[j].y, raw[j].w, 0x5410u);
          qf[t][j][2] = prmt(raw[j].x, raw[j].z, 0x7632u);
          qf[t][j][3] = prmt(raw[j].y, raw[j].w, 0x7632u);
          const float2 f0 = h2f2(raw[j].x), f1 = h2f2(raw[j].y), f2 = h2f2(raw[j].z), f3 = h2f2(raw[j].w);
          sum += ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        sum *= a.scale_log2;
        qsum[t].x = __shfl_sync(0xffffffffu, sum, 8 * c);
        qsum[t].y = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row_e = row0 + 8 * t + (kTwin ? (2 * c + e) & 3 : 2 * c + e);
          lim[t][e] = row_e < rows ? len - a.Lq + row_e / a.G : -1;
        }
      }
      const int all_see = len - a.Lq + row0 / a.G;  // tokens up to here are seen by every row of the unit

      float o[NT][kMt][4];           // fragments: rows 2c and 2c + 1 of the unit in [0, 2) and [2, 4)
      float ws[NT][4];               // sums of the signed rounded weights of rows 2c and 2c + 1 (twice)
      float2 m[NT], l[NT], vl[NT];   // of rows 2c and 2c + 1; l and vl: this thread's tokens only
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int i = 0; i < kMt; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
        m[t] = l[t] = vl[t] = both(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) ws[t][e] = 0.f;
      }
      const float c_lo = 16777216.f * a.scale_log2;
      const int tok = token_of<D>(g);  // this thread's tokens in scores: tok and tok + 8
      const int tv0 = token_of<D>(2 * c), tv1 = token_of<D>(2 * c + 1);  // in values: those and those + 8

      bool fresh = true;  // no step of this unit yet
      const uint32_t mask0 = 0x000f000fu, mask1 = 0x00f000f0u, flip0 = 0x000f0000u, flip1 = 0x00f00000u;

      // One step of two blocks of 16 tokens from t0.  kEdge: it may hold tokens that some row does not see, or that lie
      // behind the sequence (whose bytes are then whatever the page or the ring held).
      auto step = [&](auto edge_tag, const uint8_t* base, int t0) {
        constexpr bool kEdge = decltype(edge_tag)::value;
        constexpr int kB = kStep / kKvBlock;
        // ---- scores, less the running maximum ----
        float2 vp[kB][2];  // {signed s, middle of the range} of this thread's two tokens' values
        const uint32_t sign = (uint32_t)(g & 1) << 31;  // of this thread's tokens' weights
        float lmax = kNoMax, lv[kB][2];
        float sc[kB][NT][4];  // rows 2c and 2c + 1 of token tok, then of tok + 8
        bool raise = fresh;
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const uint8_t* b16 = base + b * L::kBytes;
          uint32_t kw[2][kKw];
          float kx[2], ky[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* ad = b16 + (tok + 8 * hh) * L::kRow + 4 * kKw * c;
            if constexpr (kKw == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(ad);
              kw[hh][0] = v.x, kw[hh][1] = v.y, kw[hh][2] = v.z, kw[hh][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(ad);
              kw[hh][0] = v.x, kw[hh][1] = v.y;
            }
            float2 kp = h2f2(*reinterpret_cast<const uint32_t*>(b16 + L::kKp + 4 * (tok + 8 * hh)));
            vp[b][hh] = h2f2(*reinterpret_cast<const uint32_t*>(b16 + L::kVp + 4 * (tok + 8 * hh)));
            if (kEdge && t0 + b * kKvBlock + tok + 8 * hh >= len) kp = make_float2(1.f, 0.f), vp[b][hh] = make_float2(kLeast, 0.f);
            raise |= fabsf(vp[b][hh].x) == 1.f;
            vp[b][hh].y = fmaf(7.5f, vp[b][hh].x, vp[b][hh].y);
            kx[hh] = kp.x * c_lo, ky[hh] = kp.y;
            lv[b][hh] = lg2(fmaxf(fabsf(vp[b][hh].x), kLeast));
            vp[b][hh].x = __uint_as_float(__float_as_uint(vp[b][hh].x) ^ sign);
            lmax = fmaxf(lmax, lv[b][hh]);
          }
          float lo4[NT][4], hi4[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) lo4[t][e] = hi4[t][e] = 0.f;
#pragma unroll
          for (int j = 0; j < kKw; ++j) {
            const uint32_t x = kw[0][j], y = kw[1][j], x8 = x >> 8, y8 = y >> 8;
            const uint32_t al[4] = {x & 0x000f000fu, y & 0x000f000fu, x8 & 0x000f000fu, y8 & 0x000f000fu};
            const uint32_t ah[4] = {x & 0x00f000f0u, y & 0x00f000f0u, x8 & 0x00f000f0u, y8 & 0x00f000f0u};
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma16816(lo4[t], al, qf[t][j][0], qf[t][j][1]);
              mma16816(hi4[t], ah, qf[t][j][2], qf[t][j][3]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int hh = e >> 1;
              const float q = e & 1 ? qsum[t].y : qsum[t].x, top = e & 1 ? m[t].y : m[t].x;
              const float dot = fmaf(hi4[t][e], 0.0625f, lo4[t][e]);
              sc[b][t][e] = fmaf(kx[hh], dot, fmaf(ky[hh], q, -top));
              if (kEdge && t0 + b * kKvBlock + tok + 8 * hh > lim[t][e & 1]) sc[b][t][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float top = fmaxf(fmaxf(sc[0][t][0], sc[0][t][1]), fmaxf(sc[0][t][2], sc[0][t][3]));
          top = fmaxf(top, fmaxf(fmaxf(sc[1][t][0], sc[1][t][1]), fmaxf(sc[1][t][2], sc[1][t][3])));
          raise |= top > kRaise - lmax;
        }
        if (__any_sync(0xffffffffu, raise)) {
          // tokens whose s is 1: those without codes are constant
#pragma unroll
          for (int b = 0; b < kB; ++b)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint8_t* b16 = base + b * L::kBytes;
              const bool one = fabsf(vp[b][hh].x) == 1.f;
              if (__any_sync(0xffffffffu, one) && no_codes<D>(b16 + L::kV + (tok + 8 * hh) * L::kRow) && one) {
                const float lo = h2f2(*reinterpret_cast<const uint32_t*>(b16 + L::kVp + 4 * (tok + 8 * hh))).y;
                vp[b][hh] = make_float2(__uint_as_float(__float_as_uint(kLeast) ^ sign), fmaf(7.5f, kLeast, lo));
                lv[b][hh] = kLeastLog2;
              }
            }
          __syncwarp();
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float up[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(fmaxf(sc[0][t][e] + lv[0][0], sc[0][t][e + 2] + lv[0][1]),
                              fmaxf(sc[1][t][e] + lv[1][0], sc[1][t][e + 2] + lv[1][1]));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              // the first step sets m, whatever it was; a row that sees nothing in it sees nothing later either
              up[e] = fresh && x > kNoMax ? x - kTop : fmaxf(0.f, x - kTop);
              const float f = fresh ? 1.f : ex2(-up[e]);  // sums of nothing stay zero
#pragma unroll
              for (int i = 0; i < kMt; ++i) o[t][i][e] *= f, o[t][i][e + 2] *= f;
#pragma unroll
              for (int b = 0; b < kB; ++b) sc[b][t][e] -= up[e], sc[b][t][e + 2] -= up[e];
              (e ? l[t].y : l[t].x) *= f;
              (e ? vl[t].y : vl[t].x) *= f;
              ws[t][e] *= f;
            }
            m[t].x += up[0], m[t].y += up[1];
          }
        }
        fresh = false;
        // ---- weights and values ----
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          uint32_t wb[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float w[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p = ex2(sc[b][t][2 * hh + e]);
                w[e] = p * vp[b][hh].x;
                float& vs = e ? vl[t].y : vl[t].x;
                if constexpr (kEdge) {  // what a row does not see may hold NaN
                  const bool sees = t0 + b * kKvBlock + tok + 8 * hh <= lim[t][e];
                  if (!sees) w[e] = 0.f;
                  if (sees) vs = fmaf(p, vp[b][hh].y, vs);
                } else {
                  vs = fmaf(p, vp[b][hh].y, vs);
                }
                (e ? l[t].y : l[t].x) += p;
              }
              uint32_t wr = pack_h2(w[0], w[1]);
              if constexpr (kTwin) {
                const float2 back = h2f2(wr);
                if (c >= 2) wr = pack_h2(w[0] - back.x, w[1] - back.y);
              }
              wb[t][hh] = movmatrix_trans(wr);
            }
          // codes: words 2g and 2g + 1 (D = 64: word g) of four tokens, paired by token
          uint32_t xv[2][2][2];  // [tile rows g / g + 8][token half][low / high 16 bits of the word]
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* r0 = base + b * L::kBytes + L::kV + (tv0 + 8 * hh) * L::kRow;
            const uint8_t* r1 = base + b * L::kBytes + L::kV + (tv1 + 8 * hh) * L::kRow;
            if constexpr (D == 128) {
              const uint2 p = *reinterpret_cast<const uint2*>(r0 + 8 * g), q = *reinterpret_cast<const uint2*>(r1 + 8 * g);
              xv[0][hh][0] = prmt(p.x, q.x, 0x5410u), xv[0][hh][1] = prmt(p.x, q.x, 0x7632u);
              xv[1][hh][0] = prmt(p.y, q.y, 0x5410u), xv[1][hh][1] = prmt(p.y, q.y, 0x7632u);
            } else {
              const uint32_t p = *reinterpret_cast<const uint32_t*>(r0 + 4 * g);
              const uint32_t q = *reinterpret_cast<const uint32_t*>(r1 + 4 * g);
              xv[0][hh][0] = prmt(p, q, 0x5410u), xv[1][hh][0] = prmt(p, q, 0x7632u);
            }
          }
          const uint32_t ones[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(ws[t], ones, wb[t][0], wb[t][1]);
#pragma unroll
          for (int i = 0; i < kMt; ++i) {
            // tile i: rows g and g + 8 are nibble i of the two words (D = 128), nibbles i and i + 4 of the one (64)
            const int half = D == 128 ? i >> 2 : 0;
            if (i % 4 == 2)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
                xv[0][hh][half] >>= 8, xv[1][hh][half] >>= 8;
            // the second token of a pair as 15 - code
            const uint32_t mask = i & 1 ? mask1 : mask0, flip = i & 1 ? flip1 : flip0;
            const uint32_t av[4] = {and_xor(xv[0][0][half], mask, flip), and_xor(xv[1][0][half], mask, flip),
                                    and_xor(xv[0][1][half], mask, flip), and_xor(xv[1][1][half], mask, flip)};
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(o[t][i], av, wb[t][0], wb[t][1]);
          }
        }
      };

      const int s_end = u.s + (end - at);
      for (int s = max(u.s, kLead) - kLead; s < s_end - kLead; ++s) {
        if (alive && !mbar_wait_warp(&full[slot], parity)) {
          alive = false;  // nothing is handed back from here on, so nothing more is requested
          if (lane == 0) report_error(a.err, kErrTimeoutFull);
          for (int i = 1; i < kS; ++i) {  // the other copies in flight must not outlive the kernel
            const int sl = (slot + i) % kS;
            mbar_wait_bounded(&full[sl], sl < slot ? parity ^ 1 : parity);
          }
        }
        const uint8_t* base = ring + slot * C::kStepBytes;
        const int t0 = s * kStep;
        if (t0 + kStep - 1 <= all_see)
          step(std::false_type{}, base, t0);
        else
          step(std::true_type{}, base, t0);
        fence_proxy_async_smem();  // the loads above before the copy that refills the stage
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(&empty[slot]);
        slot = slot + 1 == kS ? 0 : slot + 1;
        parity ^= slot == 0;
      }

      // ---- the unit's result, or this warp's part of it --------------------------------------------
      const bool open_left = u.s > (a.split ? 0 : kLead), open_right = at + (u.n - u.s) > r1, whole = !open_left && !open_right;
      float* dst = open_left ? join + warp * C::kRows * C::kJoinPitch : const_cast<float*>(reinterpret_cast<const float*>(ring));
      float2* mld = ml + ((open_left ? 0 : kW) + warp) * C::kRows;
      if (lane == 0 && !whole)
        (open_left ? s_first : s_last)[warp] = make_int4(u.b, u.hr, at - u.s, open_right ? kPart : kPart | kEnds);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
          l[t].x += __shfl_xor_sync(0xffffffffu, l[t].x, d);
          l[t].y += __shfl_xor_sync(0xffffffffu, l[t].y, d);
          vl[t].x += __shfl_xor_sync(0xffffffffu, vl[t].x, d);
          vl[t].y += __shfl_xor_sync(0xffffffffu, vl[t].y, d);
        }
        if (!whole && g == 0) {
          mld[8 * t + 2 * c] = make_float2(l[t].x == 0.f ? kNoMax : m[t].x, l[t].x);
          mld[8 * t + 2 * c + 1] = make_float2(l[t].y == 0.f ? kNoMax : m[t].y, l[t].y);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float add = e ? vl[t].y : vl[t].x, ls = e ? l[t].y : l[t].x, wsum = ws[t][e];
          const int row = 8 * t + 2 * c + e, r_all = row0 + row;
          const float inv = ls == 0.f ? 0.f : 1.f / ls;
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            // D = 128: rows g are channels 16 g + i, rows g + 8 channels 16 g + 8 + i; D = 64: 8 g + i and 8 g + 4 + i
            float v[kMt];
#pragma unroll
            for (int i = 0; i < kMt; ++i) {
              const float k = (i & 1) ? 1048576.f : 16777216.f;
              v[i] = fmaf(wsum, -7.5f / k, o[t][i][e + 2 * hi]) * k;
              if constexpr (kTwin) v[i] += __shfl_xor_sync(0xffffffffu, v[i], 2);  // both halves of a weight
              v[i] += add;
            }
            const int ch = (2 * g + hi) * kMt;
            if (!whole) {
              float4* d4 = reinterpret_cast<float4*>(dst + row * C::kJoinPitch + ch);
#pragma unroll
              for (int i = 0; i < kMt / 4; ++i) d4[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            } else if (r_all < rows) {
              uint32_t h[kMt / 2];
#pragma unroll
              for (int i = 0; i < kMt / 2; ++i) h[i] = pack_h2(v[2 * i] * inv, v[2 * i + 1] * inv);
              __half* y = a.out + (((long long)u.b * a.Lq + r_all / a.G) * a.Hq + head * a.G + r_all % a.G) * D + ch;
              if constexpr (kMt == 8)
                *reinterpret_cast<uint4*>(y) = make_uint4(h[0], h[1], h[2], h[3]);
              else
                *reinterpret_cast<uint2*>(y) = make_uint2(h[0], h[1]);
            }
          }
        }
      }
      at = end;
      if (at < r1) {
        u.s = u.n - 1;
        advance(a, u, 1);
      }
    }
  }  // of the warps that compute

  // ---- join the parts of the warps -----------------------------------------------------------------
  // The parts of a unit are consecutive among first(0), last(0), first(1), last(1) ..: chain c starts with the last part
  // of warp c - 1 (chain 0 with the first part of warp 0: that unit began in an earlier CTA) and goes on with the first
  // parts of warps c .. up to one that ends the unit, or to the CTA's end.
  __syncthreads();
  const int4 none = make_int4(0, 0, 0, 0);
  const int4 info_f = lane < warps ? s_first[lane] : none, info_l = lane < warps ? s_last[lane] : none;
  const unsigned has_f = __ballot_sync(0xffffffffu, info_f.w & kPart), ends_f = __ballot_sync(0xffffffffu, info_f.w & kEnds);
  const unsigned has_l = __ballot_sync(0xffffffffu, info_l.w & kPart);
  const unsigned chains = (has_l << 1) | (has_f & 1u);
  if (chains == 0) return;
  auto chain_end = [&](int ch) { return ends_f >> ch ? ch + __ffs(ends_f >> ch) - 1 : warps - 1; };  // its last warp
  float4* fac = reinterpret_cast<float4*>(smem + C::kOffFac);
  for (int i = tid; i < 2 * kW * C::kRows; i += C::kThreads) {
    const int p = i / C::kRows, row = i % C::kRows, w = p < kW ? p : p - kW;
    if (!((p < kW ? has_f : has_l) >> w & 1u)) continue;
    const int ch = p < kW ? 31 - __clz(chains & ((2u << w) - 1u)) : w + 1, w_end = chain_end(ch);
    float top = kNoMax;
    if (ch > 0) top = ml[(kW + ch - 1) * C::kRows + row].x;
#pragma unroll 4
    for (int k = ch; k <= w_end; ++k) top = fmaxf(top, ml[k * C::kRows + row].x);
    const float2 x = ml[i];
    const float f = ex2(x.x - top);
    fac[i] = make_float4(f, x.y * f, top, 0.f);
  }
  __syncthreads();
  constexpr int kPitch = D + 4;  // floats per row of a part in the workspace: O, m, l
  for (int i = tid; i < __popc(chains) * C::kRows * (D / 4); i += C::kThreads) {
    const int k = i / (C::kRows * (D / 4)), row = i / (D / 4) % C::kRows, q4 = i % (D / 4) * 4;
    unsigned rest = chains;
    for (int x = 0; x < k; ++x) rest &= rest - 1u;
    const int ch = __ffs(rest) - 1, w_end = chain_end(ch);
    const bool ends = (ends_f >> ch) != 0, whole = ch > 0 && ends;
    const int4 info = ch > 0 ? s_last[ch - 1] : s_first[0];
    const int head = (int)quot(info.y, a.rb), r_all = (info.y - head * a.RB) * C::kRows + row;
    if (r_all >= a.Lq * a.G) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
    auto add = [&](const float4& f, const float* src) {
      const float4 z = *reinterpret_cast<const float4*>(src + row * C::kJoinPitch + q4);
      x.x = fmaf(z.x, f.x, x.x), x.y = fmaf(z.y, f.x, x.y), x.z = fmaf(z.z, f.x, x.z), x.w = fmaf(z.w, f.x, x.w);
      ls += f.y;
    };
    if (ch > 0) add(fac[(kW + ch - 1) * C::kRows + row], reinterpret_cast<const float*>(smem + (ch - 1) * kS * C::kStepBytes));
#pragma unroll 4
    for (int w = ch; w <= w_end; ++w) add(fac[w * C::kRows + row], join + w * C::kRows * C::kJoinPitch);
    if (whole) {
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      __half* y = a.out + (((long long)info.x * a.Lq + r_all / a.G) * a.Hq + head * a.G + r_all % a.G) * D + q4;
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_h2(x.x * inv, x.y * inv), pack_h2(x.z * inv, x.w * inv));
    } else {
      float* p = a.part + (((long long)blockIdx.x * 2 + (ends ? 0 : 1)) * C::kRows + row) * kPitch;
      *reinterpret_cast<float4*>(p + q4) = x;
      if (q4 == 0) *reinterpret_cast<float2*>(p + D) = make_float2(fac[(ch > 0 ? kW + ch - 1 : 0) * C::kRows + row].z, ls);
    }
  }

  // ---- join the parts of the CTAs: whoever finds a unit's parts complete -----------------------------
  // The one that goes on behind the CTA's range is in the last chain, the one that began before it in chain 0.
  const bool into = (chains & 1u) != 0;
  const int last_chain = 31 - __clz(chains);
  const bool on = (ends_f >> last_chain) == 0;
  if (!into && !on) return;
  __syncthreads();
  if (tid == 0) {
    __threadfence();  // what the CTA has written, before its flags
    if (into && ends_f) set_flag(a.flag + 2 * blockIdx.x, kThere);
    if (on) set_flag(a.flag + 2 * blockIdx.x + 1, kThere);
    __threadfence();  // its flags, before it looks at others': of two CTAs at least one sees the other's
  }
  for (int side = 0; side < 2; ++side) {
    if (!(side ? on : into && ends_f != 0)) continue;
    __syncthreads();
    const int ch = side ? last_chain : 0;
    const int4 info = ch > 0 ? s_last[ch - 1] : s_first[0];
    const int n = seq_steps(a, info.x);
    const int c0 = info.z / quota, c1 = (info.z + n - 1) / quota, parts = c1 - c0 + 1;  // the unit's CTAs
    bool there = true;
    __threadfence();
    for (int i = tid; i < parts; i += C::kThreads)
      there &= flag_set(a.flag + 2 * (c0 + i) + (i < parts - 1 ? 1 : 0));
    // The last CTA to set its flag finds them all.  Others may too, if they look before that one has taken the flags
    // back; they then write the same values.
    if (!__syncthreads_and(there)) continue;
    __threadfence();
    for (int i = tid; i < parts; i += C::kThreads) set_flag(a.flag + 2 * (c0 + i) + (i < parts - 1 ? 1 : 0), 0ull);
    const int head = (int)quot(info.y, a.rb), row0 = (info.y - head * a.RB) * C::kRows;
    // one pass over the parts, kAhead of them in flight at a time: one more trip to the L2 cache for the maxima costs 1 us
    constexpr int kAhead = D == 128 ? 20 : 10;
    for (int i = tid; i < C::kRows * (D / 4); i += C::kThreads) {
      const int row = i / (D / 4), q4 = i % (D / 4) * 4, r_all = row0 + row;
      if (r_all >= a.Lq * a.G) continue;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float ls = 0.f, top = kNoMax;
      // slot 1 of the CTAs in which the unit goes on, slot 0 of the last
      const float* first = a.part + (((long long)c0 * 2 + 1) * C::kRows + row) * kPitch;
      for (int k0 = 0; k0 < parts; k0 += kAhead) {
        float2 ml2[kAhead];
        float4 z[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int n = k0 + k;
          const float* src = first + (n * 2 - (n == parts - 1 ? 1 : 0)) * (C::kRows * kPitch);
          ml2[k] = n < parts ? __ldcg(reinterpret_cast<const float2*>(src + D)) : make_float2(kNoMax, 0.f);
          z[k] = n < parts ? __ldcg(reinterpret_cast<const float4*>(src + q4)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float now = top;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) now = fmaxf(now, ml2[k].x);
        const float old = ex2(top - now);
        top = now;
        x.x *= old, x.y *= old, x.z *= old, x.w *= old, ls *= old;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float f = ex2(ml2[k].x - top);
          x.x = fmaf(z[k].x, f, x.x), x.y = fmaf(z[k].y, f, x.y), x.z = fmaf(z[k].z, f, x.z), x.w = fmaf(z[k].w, f, x.w);
          ls = fmaf(ml2[k].y, f, ls);
        }
      }
      const float inv = ls == 0.f ? 0.f : 1.f / ls;
      __half* y = a.out + (((long long)info.x * a.Lq + r_all / a.G) * a.Hq + head * a.G + r_all % a.G) * D + q4;
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_h2(x.x * inv, x.y * inv), pack_h2(x.z * inv, x.w * inv));
    }
  }
}

int row_tiles(int rows) { return rows <= 8 ? 1 : 2; }

template <int D, int NT, bool kTwin>
cudaError_t launch(const Args& a, int ctas, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_kv_i4_kernel<D, NT, kTwin>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  // The launch may start before the kernel ahead of it has ended; it waits for it before it reads anything.
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_kv_i4_kernel<D, NT, kTwin>, a);
}

}  // namespace

// Per CTA two parts of units that span CTAs, and their flags.
size_t attn_kv_i4_workspace_bytes(int B, int Lq, int Hq, int Hkv, int D) {
  const int rows = 8 * row_tiles(Lq * (Hq / Hkv));
  (void)B;
  return (size_t)num_sms() * 2 * ((size_t)rows * (D + 4) * 4 + 8);
}

cudaError_t launch_attn_kv_i4(const uint16_t* q, long long q_stride, int B, int Lq, int Hq, int Hkv, int D,
                              const uint8_t* cache, long long pages, int ps, const int* table, int width,
                              const int* kv_lens, float scale, uint16_t* out, void* workspace, unsigned* dev_err,
                              cudaStream_t s, std::string* err) {
  const int G = Hq / Hkv, nt = row_tiles(Lq * G), sms = num_sms();
  Args a;
  a.q = reinterpret_cast<const __half*>(q);
  a.q_stride = q_stride;
  a.B = B, a.Lq = Lq, a.Hq = Hq, a.Hkv = Hkv, a.G = G;
  a.RB = (Lq * G + 8 * nt - 1) / (8 * nt);
  a.cache = cache;
  a.pages = (int)pages;
  a.table = table;
  a.width = width;
  a.kv_lens = kv_lens;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.bpp = fast_div(ps / kKvBlock);
  a.rb = fast_div(a.RB);
  a.out = reinterpret_cast<__half*>(out);
  a.part = static_cast<float*>(workspace);
  a.flag = reinterpret_cast<unsigned long long*>(static_cast<uint8_t*>(workspace) +
                                                 (size_t)sms * 2 * 8 * nt * (D + 4) * sizeof(float));
  a.err = dev_err;
  a.cap = width * ps;
  // A CTA per unit where they fit the card at once and none can be long, as far as the table's width tells: nothing to join
  // between CTAs.  Otherwise an even share of all steps for every SM, but no more CTAs than the longest possible lengths
  // could use.  With a CTA per unit the longest one decides, with even shares the joins do; by the tokens of every context
  // (us, a CTA per unit / even shares):
  //                                   512        1024       1536       2048       4096       8192
  //     8 units, 8 rows, D = 128    6.2/10.8   7.9/10.7   9.9/11.0   11.1/11.1  17.4/11.3  29.8/11.9
  //   128 units, 8 rows, D = 128    6.5/13.3   8.4/14.4  10.5/15.2   11.6/17.9  18.2/22.7  31.7/34.5
  //     8 units, 16 rows, D = 128   8.9/12.9  11.3/11.7  13.5/13.2   16.8/13.4  26.6/14.0  46.4/19.2
  //     8 units, 16 rows, D = 64    7.0/10.8   8.6/11.1  10.7/11.3   11.9/11.4  18.5/12.0  31.7/13.9
  // Up to 1536 tokens it is the better plan for all of them but the third, which loses 2 % there.  Wider tables take the
  // shares: their lengths are not known here, and one long unit would cost more than the joins do.
  const long long units = (long long)B * Hkv * a.RB, most = ((long long)a.cap + kStep - 1) / kStep + kLead;
  if (units * most > INT_MAX) {
    *err = "more than 2^31 - 1 steps of 32 tokens fit the block table";
    return cudaErrorInvalidValue;
  }
  a.split = units > sms || most > kOwnSteps + kLead;
  const int ctas = (int)(!a.split ? units : units * most < sms ? units * most : sms);
  const bool twin = Lq * G <= 4;  // free columns for the rounding's rest: at the top
  if (D == 128) {
    if (twin) return launch<128, 1, true>(a, ctas, s);
    return nt == 1 ? launch<128, 1, false>(a, ctas, s) : launch<128, 2, false>(a, ctas, s);
  }
  if (twin) return launch<64, 1, true>(a, ctas, s);
  return nt == 1 ? launch<64, 1, false>(a, ctas, s) : launch<64, 2, false>(a, ctas, s);
}

}  // namespace wql
