// kv_evict_i4.cu -- leaving the least attended tokens of a paged 4-bit KV cache behind.
//
// Of the n = kv_lens[b] tokens of sequence b, each K/V head keeps min(n, budget): the last min(recent, budget) ones and, of
// the others, those with the greatest weights (of equal ones the first; a NaN counts as greater than any number).  The kept
// ones go, in their order, into the pages of row b of new_table; their numbers and weights go to kept and new_weights.
//
// One kernel, a CTA or a cluster of CTAs for each sequence and head.  A weight is a 32-bit number that orders as the weights
// do; a thread keeps some in registers, so they are read once, whatever follows.  The smallest kept
// number is found digit by digit: each digit is counted in shared memory (a warp's equal ones, as zeros come, at once), and the
// first CTA of a cluster adds up what the others have.  Then ballots and a scan over warps and CTAs give every kept token its
// place, and the warps move the rows, a block of 16 tokens at a time with all its copies in flight at once.  The search is
// latency and the move bandwidth: where there are many heads, some search while others move.
// Where a head has more tokens than its CTAs have registers for, they are read again for every digit.
//
// Bound by that chain where heads are few, and by the move where they are many: rows of 64 bytes from all over the cache, 5.2 to
// 5.5 TB/s while it lasts, after a search of about 18 us for heads of 4096 tokens.  Measured on GB300:
//   64 contexts up to 4096, half of each kept, 8 heads of 128          61 us, 3.7 TB/s over all
//   one context of 120001, 16384 kept, 8 heads of 128                  35 us
//   24 contexts up to 3001, 1777 kept, 32 heads of 64                  47 to 49 us
//   4 contexts of 1024, 960 kept, 8 heads of 128                       10 us on the GPU, 18 to 27 through the Python call
// Selecting with one CTA per head, digits of weights read again from memory, and moving in a second kernel took 124, 335, 110 and 39.
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kBits = 11, kBins = 1 << kBits;  // of a digit: 11, 11 and 10 bits

struct Args {
  const float* weights;  // [B, H, cap]
  uint8_t* cache;
  int pages, ps, H;
  FastDiv by_ps, by_bpp;
  const int* table;
  int width, cap;
  const int* kv_lens;
  int B;
  const int* new_table;
  int new_width, new_cap, budget, recent;
  int* kept;           // [B, H, budget]
  float* new_weights;  // [B, H, new_cap]
  int* new_lens;
  unsigned* err;
};

// Greater weights have greater numbers; minus zero counts as zero, a NaN as the greatest of all.
__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0xffffffffu : u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_peer(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_cluster(p, rank)) : "memory");
  return v;
}

__device__ __forceinline__ void st_peer(void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_cluster(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void red_peer(void* p, int rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(map_cluster(p, rank)), "r"(v) : "memory");
}

// Moves the rows of blocks `first`, `first` + `step` .. of 16 kept tokens of a K/V head, a warp each: 16 bytes of codes per
// lane at a time.
template <int D>
__device__ __forceinline__ void move_rows(const Args& a, int b, int h, const int* kept, int keep, int first, int step) {
  using L = KvI4<D>;
  constexpr int kChunks = 2 * L::kRow / 16;  // of 16 bytes, per token: K's, then V's
  constexpr int kIter = kKvBlock * kChunks / 32;
  const int lane = threadIdx.x & 31, bpp = a.ps / kKvBlock, blocks = keep > 0 ? (keep - 1) / kKvBlock + 1 : 0;
  // lane: where token lane % 16 of a block is, its block's offset (a multiple of 128) plus its row there; -1: nowhere
  auto source = [&](int blk) {
    if (blk >= blocks) return -1LL;
    const int i = blk * kKvBlock + (lane & 15);
    if (i >= keep) return -1LL;
    const int t = kept[i], pg = (int)quot((uint32_t)t, a.by_ps), at = t - pg * a.ps, page = a.table[(long long)b * a.width + pg];
    if (page < 0 || page >= a.pages) {
      report_error(a.err, kErrBadIndex);
      return -1LL;
    }
    return (((long long)page * a.H + h) * bpp + at / kKvBlock) * L::kBytes + at % kKvBlock;
  };
  auto target = [&](int blk) { return blk < blocks ? a.new_table[(long long)b * a.new_width + quot(blk, a.by_bpp)] : 0; };
  long long next = source(first);
  int next_to = target(first);
  for (int blk = first; blk < blocks; blk += step) {
    long long from = next;
    const int to = next_to, pb = (int)quot(blk, a.by_bpp);
    if (to < 0 || to >= a.pages) {
      report_error(a.err, kErrBadIndex);
      from = -1;
    }
    uint8_t* dst = a.cache + (((long long)to * a.H + h) * bpp + (blk - pb * bpp)) * L::kBytes;
    uint4 v[kIter];
    uint32_t par = 0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
      const long long f = __shfl_sync(0xffffffffu, from, row);
      const int r = (int)f & (kKvBlock - 1), part = ch >= kChunks / 2 ? L::kV : 0, c = ch % (kChunks / 2);
      if (f >= 0) v[i] = __ldcs(reinterpret_cast<const uint4*>(a.cache + (f - r) + part + r * L::kRow + 16 * c));
    }
    // lanes 0-15: K's parameters, 16-31: V's
    const int pr = (int)from & (kKvBlock - 1), ppart = lane < 16 ? L::kKp : L::kVp;
    if (from >= 0) par = __ldcs(reinterpret_cast<const uint32_t*>(a.cache + (from - pr) + ppart + 4 * pr));
    next = source(blk + step), next_to = target(blk + step);  // while these are under way
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
      const int part = ch >= kChunks / 2 ? L::kV : 0, c = ch % (kChunks / 2);
      if (__shfl_sync(0xffffffffu, from, row) >= 0) *reinterpret_cast<uint4*>(dst + part + row * L::kRow + 16 * c) = v[i];
    }
    if (from >= 0) *reinterpret_cast<uint32_t*>(dst + ppart + 4 * (lane & 15)) = par;
  }
}

// kPer: tokens of a thread; kCtas: of a cluster
template <int D, int kThreads, int kPer, int kCtas>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : kThreads == 512 ? 2 : 1) kv_evict_kernel(const Args a) {
  constexpr int kWarps = kThreads / 32, kStep = kThreads * kPer;
  __shared__ uint32_t hist[2][kBins];  // two digits' in turn: a CTA may still read the last one's
  __shared__ uint32_t s_warp[2][kWarps], s_pick[2][2], s_total[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kCtas > 1 ? (int)cluster_ctarank() : 0;
  const int bh = blockIdx.x / kCtas, b = bh / a.H;
  grid_dependency_wait();
  grid_dependents_launch();
  auto sync_all = [&]() {
    if (kCtas > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  int n = max(a.kv_lens[b], 0);
  if (n > a.cap) {
    if (tid == 0) report_error(a.err, kErrBadIndex);
    n = a.cap;
  }
  const int keep = min(n, a.budget), old = n - min(min(a.recent, a.budget), n);  // tokens 0 .. old - 1 compete
  const int places = keep - (n - old);                                           // of them are kept
  const float* w = a.weights + (long long)bh * a.cap;
  int* kept = a.kept + (long long)bh * a.budget;
  float* nw = a.new_weights + (long long)bh * a.new_cap;
  if (rank == 0 && tid == 0 && bh % a.H == 0) a.new_lens[b] = keep;
  const long long behind = (long long)keep + rank * kThreads + tid;  // may pass 2^31
  for (long long i = behind; i < a.budget; i += kCtas * kThreads) kept[i] = -1;
  for (long long i = behind; i < a.new_cap; i += kCtas * kThreads) nw[i] = 0.f;
  const int rounds = n > 0 ? (n - 1) / (kCtas * kStep) + 1 : 0;  // 1: all tokens are in registers
  // the tokens of a round: a warp has 32 kPer consecutive ones, 32 at a time, so that loads and stores are whole lines
  float x[kPer];
  auto load = [&](int round) {
    const uint32_t t = (((uint32_t)(round * kCtas + rank) * kWarps + warp) * kPer) * 32 + lane;  // may pass 2^31
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = t + 32 * i < (uint32_t)n ? w[t + 32 * i] : 0.f;
    return t;
  };
  uint32_t t0 = load(0);
  uint32_t prefix = 0, ties = 0;  // the smallest kept number; how many of those that have it are kept
  const bool search = places > 0 && places < old;
  if (search) {
    uint32_t need = places;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1 << 10 : kBins;
      const uint32_t mask = d == 0 ? 0u : 0xffffffffu << (d == 1 ? 21 : 10);
      uint32_t* h = hist[d & 1];
      for (int i = tid; i < kBins; i += kThreads) h[i] = 0;
      __syncthreads();
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) t0 = load(r);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t k = order_of(x[i]), bin = k >> shift & (bins - 1);
          const bool in = t0 + 32 * i < (uint32_t)old && (k & mask) == prefix;
          const unsigned lanes = __ballot_sync(0xffffffffu, in);
          if (lanes == 0) continue;
          // where all digits are the same, as those of many zeros, one lane counts them
          const uint32_t one = __shfl_sync(0xffffffffu, bin, __ffs(lanes) - 1);
          if (__all_sync(0xffffffffu, !in || bin == one)) {
            if (lane == 0) atomicAdd(&h[one], (uint32_t)__popc(lanes));
          } else if (in) {
            atomicAdd(&h[bin], 1u);
          }
        }
      }
      if (kCtas > 1) {  // the first CTA adds up the counts that there are
        cluster_sync();
        if (rank > 0)
          for (int i = tid; i < bins; i += kThreads)
            if (h[i]) red_peer(&h[i], 0, h[i]);
        cluster_sync();
      } else {
        __syncthreads();
      }
      // the bin that holds the last kept one, counting from the greatest
      constexpr int kEach = kBins / kThreads;
      uint32_t c[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int bin = bins - 1 - (tid * kEach + i);
        c[i] = bin >= 0 && rank == 0 ? h[bin] : 0u;
        sum += c[i];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
      }
      if (lane == 31) s_warp[0][warp] = incl;
      __syncthreads();
      for (int v = 0; v < warp; ++v) incl += s_warp[0][v];
      uint32_t above = incl - sum;
      if (above < need && need <= incl) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          if (above < need && need <= above + c[i]) {
#pragma unroll
            for (int p = 0; p < kCtas; ++p) {
              st_peer(&s_pick[d & 1][0], p, bins - 1 - (tid * kEach + i));
              st_peer(&s_pick[d & 1][1], p, need - above);
            }
          }
          above += c[i];
        }
      }
      sync_all();
      prefix |= s_pick[d & 1][0] << shift;
      need = s_pick[d & 1][1];
    }
    ties = need;
  }
  // counting off: how many of the tokens before are greater than the smallest kept number or too new to compete, and ties
  uint32_t done = 0, met = 0;  // of the rounds before
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) t0 = load(r);
    auto is_sure = [&](int i, uint32_t k) {
      const uint32_t t = t0 + 32 * i;
      return t < (uint32_t)n && (t >= (uint32_t)old || (search ? k > prefix : places > 0));
    };
    auto is_tie = [&](int i, uint32_t k) { return search && t0 + 32 * i < (uint32_t)old && k == prefix; };
    uint32_t mine = 0;  // of the warp: sure ones, ties in the upper half; a CTA has 2^14 tokens at most
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t k = order_of(x[i]);
      mine += __popc(__ballot_sync(0xffffffffu, is_sure(i, k))) + (__popc(__ballot_sync(0xffffffffu, is_tie(i, k))) << 16);
    }
    __syncthreads();
    if (lane == 0) s_warp[r & 1][warp] = mine;
    __syncthreads();
    uint32_t v = lane < kWarps ? s_warp[r & 1][lane] : 0u, before = lane < warp ? v : 0u;
    v = __reduce_add_sync(0xffffffffu, v), before = __reduce_add_sync(0xffffffffu, before);
    uint32_t at = done + (before & 0xffffu), ties_at = met + (before >> 16);
    if (kCtas > 1) {
      if (tid == 0) s_total[r & 1] = v;
      cluster_sync();
#pragma unroll
      for (int p = 0; p < kCtas; ++p) {
        const uint32_t o = ld_peer(&s_total[r & 1], p);
        if (p < rank) at += o & 0xffffu, ties_at += o >> 16;
        done += o & 0xffffu, met += o >> 16;
      }
    } else {
      done += v & 0xffffu, met += v >> 16;
    }
    at += min(ties_at, ties);  // of the ties before, as many are kept as there is room for
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t k = order_of(x[i]);
      const unsigned tie = __ballot_sync(0xffffffffu, is_tie(i, k));
      const bool in = is_sure(i, k) || ((tie >> lane & 1) && ties_at + __popc(tie & below) < ties);
      const unsigned all = __ballot_sync(0xffffffffu, in);
      const uint32_t to = at + __popc(all & below);
      if (in) kept[to] = (int)(t0 + 32 * i), nw[to] = x[i];
      at += __popc(all), ties_at += __popc(tie);
    }
  }
  sync_all();  // the kept tokens are all listed, and no CTA leaves while another reads its counts
  move_rows<D>(a, b, bh - b * a.H, kept, keep, rank * kWarps + warp, kCtas * kWarps);
}

template <int D, int kThreads, int kPer, int kCtas>
cudaError_t launch(const Args& a, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * a.H * kCtas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = kCtas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kv_evict_kernel<D, kThreads, kPer, kCtas>, a);
}

// The table's width, which bounds the lengths, and the number of heads decide.  A head gets as many CTAs as fit the card with those of
// all heads, two per SM, since a head's search is a chain of latencies and a single CTA moves 16 rows at a time per warp; and
// registers for all its tokens where it can, else they are read again for each digit.  On GB300, us (threads x tokens of each x CTAs,
// what the rule takes first; tokens of a head, half of them kept unless said):
//     32 heads of  1000, 900 kept   512x2x1  9.7   256x4x1 12.4   256x4x4 12.6   512x4x1 10.5
//      8 heads of  2000             512x4x1 12.8   256x16x1 22.4  512x4x4 13.4
//      8 heads of  4000             512x4x4 14.1   512x4x8 13.0   256x16x1 25.7
//     32 heads of  4000             512x4x4 14.5   512x4x8 16.5   512x4x2 16.6   256x16x1 26.5
//    128 heads of  4000             512x4x2 23.0   512x4x4 35.4   256x16x1 36.9
//    160 heads of  4000             256x16x1 41.6  512x4x1 30.5   512x4x2 40.9
//    256 heads of  4000             256x16x1 49.9  512x4x1 39.9   512x4x2 51.5
//    512 heads of  4000             256x16x1 78.8  512x4x1 82.4   512x4x2 103.3
//      8 heads of 16000             512x4x8 17.0   512x16x8 24.0  512x16x2 38.7
//    128 heads of 16000, 4000 kept  512x16x2 52.4  512x16x4 73.1  512x16x8 112.5  256x16x1 96.2
//    160 heads of 16000, 4000 kept  256x16x1 108   512x16x2 86.9  512x16x4 96.4   512x16x8 139
//    256 heads of 16000, 4000 kept  256x16x1 126   512x16x2 108   512x16x4 136
//    512 heads of 16000, 4000 kept  256x16x1 187   512x16x2 197   512x16x4 259
//     64 heads of 60000, 8000 kept  512x16x4 71.9  512x16x8 83.2  512x16x2 94.3
//    160 heads of 60000, 8000 kept  256x16x1 283   512x16x2 209   512x16x4 183
//      8 heads of 120001, 16384 kept  1024x16x8 34.4  512x16x8 46.6
// Above 4096 tokens eight CTAs go to a head where they fit, below that four, since 32 heads lose more by eight than 8 heads win.  From 153
// to some 400 heads the rule's single CTA is not the best: a head with more tokens than its registers hold reads them four times.
template <int D>
cudaError_t launch(const Args& a, cudaStream_t s) {
  const long long heads = (long long)a.B * a.H, room = 2LL * num_sms();
  if (a.cap <= 1024) return heads <= room ? launch<D, 512, 2, 1>(a, s) : launch<D, 256, 4, 1>(a, s);
  if (a.cap <= 2048) return launch<D, 512, 4, 1>(a, s);
  if (heads * 8 <= room && a.cap > 4096) {
    if (a.cap <= 16384) return launch<D, 512, 4, 8>(a, s);
    return a.cap <= 65536 ? launch<D, 512, 16, 8>(a, s) : launch<D, 1024, 16, 8>(a, s);
  }
  if (heads * 4 <= room) return a.cap <= 8192 ? launch<D, 512, 4, 4>(a, s) : launch<D, 512, 16, 4>(a, s);
  if (heads * 2 <= room) return a.cap <= 4096 ? launch<D, 512, 4, 2>(a, s) : launch<D, 512, 16, 2>(a, s);
  return launch<D, 256, 16, 1>(a, s);
}

}  // namespace

cudaError_t launch_kv_evict_i4(const float* weights, uint8_t* cache, long long pages, int ps, int H, int D, const int* table,
                               int width, const int* kv_lens, int B, const int* new_table, int new_width, int budget,
                               int recent, int* kept, float* new_weights, int* new_lens, unsigned* dev_err, cudaStream_t s) {
  Args a{weights, cache, (int)pages, ps, H, fast_div(ps), fast_div(ps / kKvBlock), table, width, width * ps, kv_lens, B,
         new_table, new_width, new_width * ps, budget, recent, kept, new_weights, new_lens, dev_err};
  return D == 128 ? launch<128>(a, s) : launch<64>(a, s);
}

}  // namespace wql
