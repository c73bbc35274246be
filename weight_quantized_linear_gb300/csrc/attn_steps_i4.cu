// attn_steps_i4.cu -- attention over the paged 4-bit KV cache for chunks of a few rows: single tokens, drafted ones.
//
// attention_chunks_kv_i4's formulas for the sequences whose rows of a K/V head, tokens times query heads, are 8 NT or fewer.
// Rows are the narrow side of mma.sync products here, keys and channels the wide one:
//   S^T (16 keys x 8 rows) = K Q^T, then O^T (16 channels x 8 rows) += V^T P,
// with K and V converted from codes in registers and rounded to fp16, as the formulas ask.  A product's inner indices may be in any
// order as long as both operands agree: a thread takes its key's codes as they lie in a word, (0, 4), (1, 5) .., and Q's channels
// are put into that order once; for V two keys' words are merged by halves first, so that the same masks yield pairs of keys.
// Both products leave rows 2c and 2c + 1 in the threads that hold lane % 4 = c, so the maximum, the sum and the rescaling of the
// accumulator need an exchange only when a weight passes 2^15 and at the end.
//
// A unit is a sequence and K/V head, a step 32 of its keys.  The steps of all units, in order, are divided evenly over the
// CTAs, one per SM, and a CTA's over its warps, each a run with a ring of copies of its own, which a lane of one more warp
// keeps filled.  A unit's parts are joined in shared memory at the CTA's end, those of CTAs by the joining kernel.
//
// Bound by instructions: about 360 per warp and 16 keys of heads of 128 (208 of them masks, subtractions and multiply-adds that
// make numbers of codes, 16 products), 59 % of the issue slots used, DRAM at half its rate.  mma.sync, not tcgen05: its operands
// come out of registers, and they use a fifth of its rate.  Measured on GB300 through the Python call, or in a graph (g):
//   64 single tokens over up to 8192 (290 MB), 32 / 8 heads of 128          76 us, 3.8 TB/s, 75 g (in 128-row tiles 197)
//   4 drafted tokens x 32 over up to 6000, 32 / 8 heads of 64 (57 MB)       35 us g (76)
//   64 single tokens over up to 5000 of 16 heads per K/V head of 128 (88 MB)   49 us g
//   one row of 700 tokens, 32 heads of 128                                  11.6 us g, latency of two launches
// attention_kv_i4, which takes all sequences' rows alike, does not round the values and gives no lse, takes 59, 32, 40 and 7.5 g.
// Eight rows where they are enough: with the products for sixteen the first of these takes 100 us.
//
// Roundings: weights are fp16, as V is by the formula, sums fp32 of weights before they are rounded.  Outputs are off by 2.6e-4 of
// their norm, of which 2.1e-4 is their own rounding.  For up to four rows that could be all: the columns that they leave free
// would take what the weights' rounding leaves, as in attention_kv_i4.  Here that would cost 64 single tokens 78 us for 75 (heads of 64: 58
// for 57) and, by its branch, eight rows 78 for 77, for an error far below that of values in four bits.
#include <atomic>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "attn_chunks.cuh"
#include "internal.h"

namespace wql {
namespace {

constexpr int kStep = 32;  // keys
constexpr int kLead = 3;   // steps that stand for a unit's own cost
constexpr float kNoMax = -3e38f;
// a weight beyond 2^15 asks for a new maximum, which then has the weight 2^7
constexpr float kTop = 7.0f, kRaise = 15.0f;

template <int D, int NT>  // NT: rows by eight
struct Cfg {
  static constexpr int kRows = 8 * NT;
  // As many as registers and rings allow.  Heads of 128: 15 warps with 128 registers and two stages take 80 us for 76 (64 single
  // tokens), nine with four stages 87; heads of 64: 13 warps 69 us for 65, 11 68.
  static constexpr int kWarps = D == 128 ? 11 : 15, kThreads = 32 * (kWarps + 1);
  static constexpr int kStepBytes = kStep / kKvBlock * KvI4<D>::kBytes;
  static constexpr int kStages = D == 64 ? 4 : NT == 1 ? 3 : 2;
  static constexpr int kPitch = D + 4;                                          // floats per row of a part
  static constexpr int kOffJoin = kWarps * kStages * kStepBytes;                // [kWarps][rows][kPitch]: first parts
  static constexpr int kOffMl = kOffJoin + kWarps * kRows * kPitch * 4;      // [first, last part][kWarps][rows] {m, l}
  static constexpr int kOffFac = kOffMl + 2 * kWarps * kRows * 8;            // the same: {factor, its l, maximum}
  static constexpr int kOffBar = kOffFac + 2 * kWarps * kRows * 16;          // [full, empty][kWarps][kStages]
  static constexpr int kSmem = kOffBar + 2 * kWarps * kStages * 8;
  static_assert(kRows * kPitch * 4 <= kStages * kStepBytes, "a last part takes the warp's ring");
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16).
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ KvChunk chunk(const StepArgs& a, int b, unsigned* err = nullptr) {
  return kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, err);
}
// Steps of a unit, the first kLead of which are no keys; one with none where there are no keys.  0: not taken here.
__device__ __forceinline__ int unit_steps(const StepArgs& a, const KvChunk& k) {
  return k.rows < 1 || k.rows > a.few ? 0 : (k.len > 0 ? (k.len - 1) / kStep + 1 : 1) + kLead;
}

// Position in the order of all steps: sequence, K/V head, step s of `n` of that unit.
struct Cursor {
  int b, h, s, n;
};
__device__ __forceinline__ void advance(const StepArgs& a, Cursor& c, int by) {
  c.s += by;
  while (c.s >= c.n) {
    c.s -= c.n;
    if (++c.h == a.Hkv) {
      c.h = 0;
      do {
        if (++c.b >= a.B) {
          c.n = INT_MAX;  // past the end: nothing is read there
          return;
        }
        c.n = unit_steps(a, chunk(a, c.b));
      } while (c.n == 0);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) attn_steps_i4_kernel(const StepArgs a) {
  using C = Cfg<D, NT>;
  using L = KvI4<D>;
  constexpr int kW = C::kWarps, kS = C::kStages;
  constexpr int kKw = D / 32;  // words of K codes per thread and key
  constexpr int kMt = D / 16;  // 16-channel tiles of the output
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + C::kOffJoin);
  float2* ml = reinterpret_cast<float2*>(smem + C::kOffMl);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  __shared__ Cursor s_start[kW];            // the warps' first positions
  __shared__ int4 s_first[kW], s_last[kW];  // {sequence, head, -, kPart | kEnds}
  __shared__ long long s_sum[kW + 1];
  constexpr int kPart = 1, kEnds = 2;       // there is such a part; the unit ends in it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  for (int i = tid; i < 2 * kW * kS; i += C::kThreads) mbar_init(&bars[i], 1);
  fence_mbarrier_init();
  // Everything before this line overlaps the end of the preceding kernel.  Nothing is read before it, also where that is the kernel
  // for the other sequences: that it waited for what came before does not make it visible here.
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- this CTA's range [n0, n1) of the order of all steps; warp w's run is [run(w), run(w + 1)) ----
  long long n0, n1;
  {
    const int per = (a.B + C::kThreads - 1) / C::kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += (long long)unit_steps(a, chunk(a, b, blockIdx.x == 0 ? a.err : nullptr)) * a.Hkv;
    long long incl = mine, total = 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (warp < kW && lane == 0) s_first[warp] = s_last[warp] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int w = 0; w <= kW; ++w) {
      if (w < warp) incl += s_sum[w];
      total += s_sum[w];
    }
    // at least a step for every warp: a short batch uses fewer CTAs and has fewer parts to join
    const long long quota = max((total + gridDim.x - 1) / gridDim.x, (long long)kW);
    n0 = min(quota * blockIdx.x, total), n1 = min(n0 + quota, total);
    long long at = incl - mine;
    const long long each = (n1 - n0 + kW - 1) / kW;
    if (at < n1 && n0 < incl)
      for (int b = b0; b < b1; ++b) {
        const int n = unit_steps(a, chunk(a, b));
        const long long end = at + (long long)n * a.Hkv;
        for (int w = 0; w < kW; ++w) {
          const long long first = n0 + each * w;
          if (at <= first && first < end && first < n1) {
            const long long off = first - at;
            s_start[w] = {b, (int)(off / n), (int)(off % n), n};
          }
        }
        at = end;
      }
  }
  if (n0 >= n1) {
    if (tid == 0) a.parts.begun[blockIdx.x] = make_int4(0, 0, 0, 0), a.parts.went_on[blockIdx.x] = 0;
    return;
  }
  const long long each = (n1 - n0 + kW - 1) / kW;
  const int warps = (int)((n1 - n0 + each - 1) / each);  // with a run
  auto run = [&](int w) { return min(n0 + each * w, n1); };
  __syncthreads();

  if (warp == kW) {
    // ---------------- lane w keeps warp w's ring filled ----------------
    if (lane < warps) {
      const int bpp = (int)a.bpp.d;
      const uint32_t ring = smem_u32(smem) + lane * kS * C::kStepBytes;
      uint64_t* full = bars + lane * kS;
      uint64_t* empty = bars + (kW + lane) * kS;
      Cursor p = s_start[lane];
      long long left = run(lane + 1) - run(lane);
      int slot = 0, pg0 = 0, pg1 = 0, blk = 0, col0 = 0, last = 0, cur = -1, len = 0;
      uint32_t parity = 1;  // the first round finds every stage free
      auto next = [&](int by) {  // to the next step with keys, and the pages of its two blocks
        left -= by;
        if (by && left > 0) advance(a, p, by);
        while (left > 0 && p.s < kLead) {
          left -= 1;
          if (left > 0) advance(a, p, 1);
        }
        if (left <= 0) return;
        if (p.b != cur) cur = p.b, len = chunk(a, cur).len;
        blk = (p.s - kLead) * (kStep / kKvBlock), last = len > 0 ? (len - 1) / kKvBlock : -1;
        col0 = (int)quot((uint32_t)blk, a.bpp);
        const int* row = a.table + (long long)p.b * a.width;
        pg0 = blk <= last ? row[col0] : 0;
        pg1 = blk < last ? row[quot((uint32_t)blk + 1, a.bpp)] : pg0;
      };
      next(0);
      unsigned long long since = globaltimer_ns();
      while (left > 0) {
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
        const int in0 = blk - col0 * bpp, in1 = in0 + 1 < bpp ? in0 + 1 : 0;
        const bool two = blk < last;
        const uint32_t dst = ring + slot * C::kStepBytes;
        const uint8_t* s0 = a.cache + (((long long)pg0 * a.Hkv + p.h) * bpp + in0) * L::kBytes;
        if (last < 0) {
          mbar_arrive(&full[slot]);
        } else {
          mbar_arrive_expect_tx(&full[slot], two ? 2 * L::kBytes : L::kBytes);
          bulk_load(dst, s0, two && in1 > 0 ? 2 * L::kBytes : L::kBytes, &full[slot]);
          if (two && in1 == 0)
            bulk_load(dst + L::kBytes, a.cache + ((long long)pg1 * a.Hkv + p.h) * bpp * L::kBytes, L::kBytes, &full[slot]);
        }
        slot = slot + 1 == kS ? 0 : slot + 1;
        parity ^= slot == 0;
        next(1);
        since = globaltimer_ns();
      }
    }
  } else {
    // ---------------- the units of a warp's run ----------------
    const uint8_t* ring = smem + warp * kS * C::kStepBytes;
    uint64_t* full = bars + warp * kS;
    uint64_t* empty = bars + (kW + warp) * kS;
    int slot = 0;
    uint32_t parity = 0;
    bool alive = true;
    long long at = run(warp);
    const long long r1 = run(warp + 1);
    const float cs = a.scale_log2;
    const int tok = token_of<D>(g);  // this thread's keys in scores: tok and tok + 8; in values: two neighbours, and those + 8
    const bool swap = token_of<D>(2 * c) & 1;
    const uint32_t sel_s = swap ? 0x1054u : 0x5410u, sel_lo = swap ? 0x3276u : 0x7632u;
    Cursor u = at < r1 ? s_start[warp] : Cursor{0, 0, 0, 0};
    while (at < r1) {
      const int here = (int)min((long long)(u.n - u.s), r1 - at);  // steps of this warp's part of the unit
      const KvChunk k = chunk(a, u.b);
      const int rows = k.rows * a.G;
      // Q: thread (g, c) holds row g's channels of its K words, paired as the codes will be
      uint32_t qf[NT][kKw][4];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int row = 8 * t + g, r = row / a.G;
        const __half* src = a.q + (long long)(k.start + r) * a.q_stride + (long long)(u.h * a.G + row - r * a.G) * D + 8 * kKw * c;
        uint4 raw[kKw];
#pragma unroll
        for (int j = 0; j < kKw; ++j)
          raw[j] = row < rows ? __ldg(reinterpret_cast<const uint4*>(src) + j) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < kKw; ++j) {
          qf[t][j][0] = prmt(raw[j].x, raw[j].z, 0x5410u), qf[t][j][1] = prmt(raw[j].x, raw[j].z, 0x7632u);
          qf[t][j][2] = prmt(raw[j].y, raw[j].w, 0x5410u), qf[t][j][3] = prmt(raw[j].y, raw[j].w, 0x7632u);
        }
      }
      int lim[NT][2];           // the last keys that rows 2c and 2c + 1 see
      float o[NT][kMt][4];      // rows 2c and 2c + 1 in [0, 2) and [2, 4)
      float m[NT][2], l[NT][2]; // l: of this thread's keys
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * t + 2 * c + e;
          lim[t][e] = row < rows ? k.first + row / a.G : -1;
          m[t][e] = kNoMax, l[t][e] = 0.f;
#pragma unroll
          for (int i = 0; i < kMt; ++i) o[t][i][e] = o[t][i][e + 2] = 0.f;
        }

      // Two blocks of 16 keys from t0.  kCareful: some row may not see them all, or some parameters are infinite, not a number
      // or so large that a value may be.
      auto step = [&](auto careful, const uint8_t* base, int t0) {
        constexpr bool kCareful = decltype(careful)::value;
        constexpr int kB = kStep / kKvBlock;
        float s[kB][NT][4];  // rows 2c and 2c + 1 of key tok, then of tok + 8
        int bad = INT_MAX;   // the first of this thread's keys whose row of V is not a number
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const uint8_t* blk = base + b * L::kBytes;
          const int left = k.len - t0 - b * kKvBlock;  // keys from this block on
          uint32_t kw[2][kKw], s2[2], lo2[2];
          float acc[NT][2][4] = {};
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t ad = smem_u32(blk + (tok + 8 * hh) * L::kRow + 4 * kKw * c);
            if constexpr (kKw == 4) {
              const uint4 v = lds_u128(ad);
              kw[hh][0] = v.x, kw[hh][1] = v.y, kw[hh][2] = v.z, kw[hh][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(blk + (tok + 8 * hh) * L::kRow + 4 * kKw * c);
              kw[hh][0] = v.x, kw[hh][1] = v.y;
            }
            uint32_t par = *reinterpret_cast<const uint32_t*>(blk + L::kKp + 4 * (tok + 8 * hh));
            if constexpr (kCareful) {
              if (tok + 8 * hh >= left) par = 0u;
              if (!kv_finite(par)) par = 0x7fff7fffu;
              if (!kv_finite(*reinterpret_cast<const uint32_t*>(blk + L::kVp + 4 * (tok + 8 * hh))))
                bad = min(bad, t0 + b * kKvBlock + tok + 8 * hh);
            }
            s2[hh] = prmt(par, 0, 0x1010), lo2[hh] = prmt(par, 0, 0x3232);
          }
#pragma unroll
          for (int j = 0; j < kKw; ++j) {
            uint32_t x[4], y[4];
            kv_values8(kw[0][j], s2[0], lo2[0], x);
            kv_values8(kw[1][j], s2[1], lo2[1], y);
            if constexpr (kCareful)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = kv_clamp2(x[e]), y[e] = kv_clamp2(y[e]);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma(acc[t][0], x[0], y[0], x[1], y[1], qf[t][j][0], qf[t][j][1]);
              mma(acc[t][1], x[2], y[2], x[3], y[3], qf[t][j][2], qf[t][j][3]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // rounded before the maximum is subtracted, so that the largest has the weight 2^7 whatever it is
              s[b][t][e] = __fmul_rn(acc[t][0][e] + acc[t][1][e], cs);
              if (kCareful && t0 + b * kKvBlock + tok + 8 * (e >> 1) > lim[t][e & 1]) s[b][t][e] = -INFINITY;
            }
        }
        float up = -INFINITY;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            up = fmaxf(up, fmaxf(fmaxf(s[0][t][e], s[0][t][e + 2]), fmaxf(s[1][t][e], s[1][t][e + 2])) - m[t][e]);
        if (__any_sync(0xffffffffu, up > kRaise)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // only the rows that ask for it
              float x = fmaxf(fmaxf(s[0][t][e], s[0][t][e + 2]), fmaxf(s[1][t][e], s[1][t][e + 2]));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              const float now = x - m[t][e] > kRaise ? x - kTop : m[t][e], f = ex2(m[t][e] - now);
              m[t][e] = now, l[t][e] *= f;
#pragma unroll
              for (int i = 0; i < kMt; ++i) o[t][i][e] *= f, o[t][i][e + 2] *= f;
            }
        }
#pragma unroll
        for (int b = 0; b < kB; ++b) {
          const uint8_t* blk = base + b * L::kBytes;
          uint32_t w[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float p0 = ex2(s[b][t][2 * hh] - m[t][0]), p1 = ex2(s[b][t][2 * hh + 1] - m[t][1]);
              l[t][0] += p0, l[t][1] += p1;
              w[t][hh] = movmatrix_trans(pack_h2(p0, p1));
            }
          // words 2g and 2g + 1 (D = 64: word g) of four keys, paired by key: low and high halves
          uint32_t xv[2][2][D / 64], s2[2], lo2[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint8_t* r0 = blk + L::kV + (token_of<D>(2 * c) + 8 * hh) * L::kRow;
            const uint8_t* r1 = blk + L::kV + (token_of<D>(2 * c + 1) + 8 * hh) * L::kRow;
            if constexpr (D == 128) {
              const uint2 p = *reinterpret_cast<const uint2*>(r0 + 8 * g), q = *reinterpret_cast<const uint2*>(r1 + 8 * g);
              xv[0][hh][0] = prmt(p.x, q.x, 0x5410u), xv[0][hh][1] = prmt(p.x, q.x, 0x7632u);
              xv[1][hh][0] = prmt(p.y, q.y, 0x5410u), xv[1][hh][1] = prmt(p.y, q.y, 0x7632u);
            } else {
              const uint32_t p = *reinterpret_cast<const uint32_t*>(r0 + 4 * g), q = *reinterpret_cast<const uint32_t*>(r1 + 4 * g);
              xv[0][hh][0] = prmt(p, q, 0x5410u), xv[1][hh][0] = prmt(p, q, 0x7632u);
            }
            uint2 par = *reinterpret_cast<const uint2*>(blk + L::kVp + 4 * (2 * c + 8 * hh));
            if constexpr (kCareful) {
              const int t = t0 + b * kKvBlock + 2 * c + 8 * hh;
              if (!kv_finite(par.x) || t >= k.len) par.x = 0u;
              if (!kv_finite(par.y) || t + 1 >= k.len) par.y = 0u;
            }
            s2[hh] = prmt(par.x, par.y, sel_s), lo2[hh] = prmt(par.x, par.y, sel_lo);
          }
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t v[2][2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                kv_values8(xv[r][hh][i], s2[hh], lo2[hh], v[r][hh]);
                if constexpr (kCareful)
#pragma unroll
                  for (int e = 0; e < 4; ++e) v[r][hh][e] = kv_clamp2(v[r][hh][e]);
              }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(o[t][4 * i + e], v[0][0][e], v[1][0][e], v[0][1][e], v[1][1][e], w[t][0], w[t][1]);
          }
        }
        if constexpr (kCareful) {  // rows that see a row of V that is not a number
          bad = __reduce_min_sync(0xffffffffu, bad);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (bad <= lim[t][e])
#pragma unroll
                for (int i = 0; i < kMt; ++i) o[t][i][e] = o[t][i][e + 2] = __uint_as_float(0x7fc00000u);
        }
      };

      for (int st = max(u.s, kLead) - kLead; st < u.s + here - kLead; ++st) {
        if (alive && !mbar_wait_warp(&full[slot], parity)) {
          alive = false;  // nothing is handed back from here on, so nothing more is requested
          if (lane == 0) report_error(a.err, kErrTimeoutFull);
          for (int i = 1; i < kS; ++i) {  // the other copies in flight must not outlive the kernel
            const int sl = (slot + i) % kS;
            mbar_wait_bounded(&full[sl], sl < slot ? parity ^ 1 : parity);
          }
        }
        const uint8_t* base = ring + slot * C::kStepBytes;
        const int t0 = st * kStep;
        // parameters that could make a value of 2^15 or more: |s| from 2^11, |lo| from 2^14
        uint32_t odd = 0;
#pragma unroll
        for (int b = 0; b < kStep / kKvBlock; ++b)
          odd |= (*reinterpret_cast<const uint32_t*>(base + b * L::kBytes + L::kKp + 4 * lane) & 0x7fff7fffu) + 0x0c001800u;
        if (t0 + kStep - 1 <= k.first && !__any_sync(0xffffffffu, odd & 0x80008000u))
          step(std::false_type{}, base, t0);
        else
          step(std::true_type{}, base, t0);
        fence_proxy_async_smem();  // the loads above before the copy that refills the stage
        __syncwarp();
        if (alive && lane == 0) mbar_arrive(&empty[slot]);
        slot = slot + 1 == kS ? 0 : slot + 1;
        parity ^= slot == 0;
      }

      // ---- the unit's result, or this warp's part of it ----
      const bool open_left = u.s > 0, open_right = here < u.n - u.s, whole = !open_left && !open_right;
      float* dst = open_left ? join + warp * C::kRows * C::kPitch : const_cast<float*>(reinterpret_cast<const float*>(ring));
      float2* mld = ml + ((open_left ? 0 : kW) + warp) * C::kRows;
      if (lane == 0 && !whole) (open_left ? s_first : s_last)[warp] = make_int4(u.b, u.h, 0, open_right ? kPart : kPart | kEnds);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
          const int row = 8 * t + 2 * c + e, r = row / a.G;
          const float inv = lim[t][e] < 0 ? 0.f : 1.f / l[t][e];
          const long long to = (long long)(k.start + r) * a.Hq + u.h * a.G + row - r * a.G;
          if (!whole && g == 0) mld[row] = make_float2(m[t][e], l[t][e]);
          if (whole && g == 0 && row < rows && a.lse)
            a.lse[to] = lim[t][e] < 0 ? -INFINITY : (m[t][e] + lg2(l[t][e])) * 0.6931471805599453f;
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            // D = 128: rows g of tile i are channels 16 g + i, rows g + 8 channels 16 g + 8 + i; D = 64: 8 g + i and 8 g + 4 + i
            const int ch = (2 * g + hi) * kMt, x = e + 2 * hi;
            if (!whole) {
              float4* d4 = reinterpret_cast<float4*>(dst + row * C::kPitch + ch);
#pragma unroll
              for (int i = 0; i < kMt / 4; ++i)
                d4[i] = make_float4(o[t][4 * i][x], o[t][4 * i + 1][x], o[t][4 * i + 2][x], o[t][4 * i + 3][x]);
            } else if (row < rows) {
              uint32_t h[kMt / 2];
#pragma unroll
              for (int i = 0; i < kMt / 2; ++i) h[i] = pack_h2(o[t][2 * i][x] * inv, o[t][2 * i + 1][x] * inv);
              __half* y = a.out + to * D + ch;
              if constexpr (kMt == 8)
                *reinterpret_cast<uint4*>(y) = make_uint4(h[0], h[1], h[2], h[3]);
              else
                *reinterpret_cast<uint2*>(y) = make_uint2(h[0], h[1]);
            }
          }
        }
      at += here;
      if (at < r1) {
        u.s = u.n - 1;
        advance(a, u, 1);
      }
    }
  }

  // ---- the parts of the warps ----
  // The parts of a unit are consecutive among first(0), last(0), first(1), last(1) ..: chain i starts with the last part
  // of warp i - 1 (chain 0 with the first part of warp 0: that unit began in an earlier CTA) and goes on with the first
  // parts of warps i .. up to one that ends the unit, or to the CTA's end.
  __syncthreads();
  const int4 none = make_int4(0, 0, 0, 0);
  const int4 info_f = lane < warps ? s_first[lane] : none, info_l = lane < warps ? s_last[lane] : none;
  const unsigned has_f = __ballot_sync(0xffffffffu, info_f.w & kPart), ends_f = __ballot_sync(0xffffffffu, info_f.w & kEnds);
  const unsigned has_l = __ballot_sync(0xffffffffu, info_l.w & kPart);
  const unsigned chains = (has_l << 1) | (has_f & 1u);
  auto chain_end = [&](int ch) { return ends_f >> ch ? ch + __ffs(ends_f >> ch) - 1 : warps - 1; };  // its last warp
  if (tid == 0) {
    const int last = chains ? 31 - __clz(chains) : 0;
    int4 begun = none;
    if (last > 0 && (ends_f >> last) == 0) {
      const KvChunk k = chunk(a, s_last[last - 1].x);
      begun = make_int4(k.start, k.rows, k.first, s_last[last - 1].y);
    }
    a.parts.begun[blockIdx.x] = begun;
    a.parts.went_on[blockIdx.x] = chains & 1u ? (ends_f ? 2 : 1) : 0;
  }
  if (chains == 0) return;
  float4* fac = reinterpret_cast<float4*>(smem + C::kOffFac);
  for (int i = tid; i < 2 * kW * C::kRows; i += C::kThreads) {
    const int p = i / C::kRows, row = i % C::kRows, w = p < kW ? p : p - kW;
    if (!((p < kW ? has_f : has_l) >> w & 1u)) continue;
    const int ch = p < kW ? 31 - __clz(chains & ((2u << w) - 1u)) : w + 1, w_end = chain_end(ch);
    float top = kNoMax;
    if (ch > 0) top = ml[(kW + ch - 1) * C::kRows + row].x;
#pragma unroll 4
    for (int w2 = ch; w2 <= w_end; ++w2) top = fmaxf(top, ml[w2 * C::kRows + row].x);
    const float2 x = ml[i];
    const float f = ex2(x.x - top);
    fac[i] = make_float4(f, x.y * f, top, 0.f);
  }
  __syncthreads();
  for (int i = tid; i < __popc(chains) * C::kRows * (D / 4); i += C::kThreads) {
    const int n = i / (C::kRows * (D / 4)), row = i / (D / 4) % C::kRows, q4 = i % (D / 4) * 4;
    unsigned rest = chains;
    for (int x = 0; x < n; ++x) rest &= rest - 1u;
    const int ch = __ffs(rest) - 1, w_end = chain_end(ch);
    const bool whole = ch > 0 && (ends_f >> ch) != 0;
    const int4 info = ch > 0 ? s_last[ch - 1] : s_first[0];
    const KvChunk k = chunk(a, info.x);
    if (row >= k.rows * a.G) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f, top = kNoMax;
    auto add = [&](const float4& f, const float* src) {
      const float4 z = *reinterpret_cast<const float4*>(src + row * C::kPitch + q4);
      x.x = fmaf(z.x, f.x, x.x), x.y = fmaf(z.y, f.x, x.y), x.z = fmaf(z.z, f.x, x.z), x.w = fmaf(z.w, f.x, x.w);
      ls += f.y, top = f.z;
    };
    if (ch > 0) add(fac[(kW + ch - 1) * C::kRows + row], reinterpret_cast<const float*>(smem + (ch - 1) * kS * C::kStepBytes));
#pragma unroll 4
    for (int w = ch; w <= w_end; ++w) add(fac[w * C::kRows + row], join + w * C::kRows * C::kPitch);
    if (whole) {
      const int r = row / a.G;
      const bool blind = k.first + r < 0;  // sees nothing
      const float inv = blind ? 0.f : 1.f / ls;
      const long long to = (long long)(k.start + r) * a.Hq + info.y * a.G + row - r * a.G;
      *reinterpret_cast<uint2*>(a.out + to * D + q4) = make_uint2(pack_h2(x.x * inv, x.y * inv), pack_h2(x.z * inv, x.w * inv));
      if (q4 == 0 && a.lse) a.lse[to] = blind ? -INFINITY : (top + lg2(ls)) * 0.6931471805599453f;
    } else {
      const long long to = ((long long)blockIdx.x * 2 + (ch > 0)) * a.parts.rows + row;
      *reinterpret_cast<float4*>(a.parts.part + to * D + q4) = x;
      if (q4 == 0) a.parts.ml[to] = make_float2(top, ls);
    }
  }
}

template <int D, int NT>
cudaError_t launch(const StepArgs& a, int ctas, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static std::atomic<bool> ready[64];  // per device; racing first calls set the same attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_steps_i4_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
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
  return cudaLaunchKernelEx(&cfg, attn_steps_i4_kernel<D, NT>, a);
}

}  // namespace

cudaError_t launch_attn_steps_i4(const StepArgs& a, int D, int ctas, cudaStream_t s) {
  if (a.few * a.G <= 8) return D == 128 ? launch<128, 1>(a, ctas, s) : launch<64, 1>(a, ctas, s);
  return D == 128 ? launch<128, 2>(a, ctas, s) : launch<64, 2>(a, ctas, s);
}

}  // namespace wql
