// kv_evict_i4.cu -- leaving the least attended tokens of a paged 4-bit KV cache behind.
//
// Of the n = kv_lens[b] tokens of sequence b, each K/V head keeps min(n, budget): the last min(recent, budget) ones and, of
// the others, those with the greatest weights (of equal ones the first; a NaN counts as greater than any number).  The kept
// ones go, in their order, into the pages of row b of new_table; their numbers and weights go to kept and new_weights.
//
// One kernel, a CTA or a cluster of CTAs for each sequence and head.  A weight is a 32-bit number that orders as the weights
// do; a thread keeps its run of consecutive ones in registers, so they are read once, whatever follows.  The smallest kept
// number is found digit by digit: each digit is counted in shared memory (a run of equal ones, as zeros come, at once) and the
// CTAs add up their counts through distributed shared memory.  Then a scan over threads and CTAs gives every kept token its
// place, and the warps move the rows, a block of 16 tokens at a time with all its copies in flight at once.  The search is
// latency and the move bandwidth: where there are many heads, some search while others move.
// Where a head has more tokens than its CTAs have registers for, they are read again for every digit.
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

// Moves the rows of blocks `first`, `first` + `step` .. of 16 kept tokens of a K/V head, a warp each: 16 bytes of codes per
// lane at a time.
template <int D>
__device__ __forceinline__ void move_rows(const Args& a, int b, int h, const int* kept, int keep, int first, int step) {
  using L = KvI4<D>;
  constexpr int kChunks = 2 * L::kRow / 16;  // of 16 bytes, per token: K's, then V's
  constexpr int kIter = kKvBlock * kChunks / 32;
  const int lane = threadIdx.x & 31, bpp = a.ps / kKvBlock;
  for (int blk = first; blk * kKvBlock < keep; blk += step) {
    const int cnt = min(keep - blk * kKvBlock, kKvBlock);
    const int pb = (int)quot(blk, a.by_bpp), to = a.new_table[(long long)b * a.new_width + pb];
    long long from = -1;  // lane: where token lane % 16 is, its block's offset (a multiple of 128) plus its row there
    if ((lane & 15) < cnt) {
      const int t = kept[blk * kKvBlock + (lane & 15)];
      const int pg = (int)quot((uint32_t)t, a.by_ps), at = t - pg * a.ps, page = a.table[(long long)b * a.width + pg];
      if (page < 0 || page >= a.pages)
        report_error(a.err, kErrBadIndex);
      else
        from = (((long long)page * a.H + h) * bpp + at / kKvBlock) * L::kBytes + at % kKvBlock;
    }
    if (to < 0 || to >= a.pages) {
      report_error(a.err, kErrBadIndex);
      continue;
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
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int row = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
      const int part = ch >= kChunks / 2 ? L::kV : 0, c = ch % (kChunks / 2);
      if (__shfl_sync(0xffffffffu, from, row) >= 0) *reinterpret_cast<uint4*>(dst + part + row * L::kRow + 16 * c) = v[i];
    }
    if (from >= 0) *reinterpret_cast<uint32_t*>(dst + ppart + 4 * (lane & 15)) = par;
  }
}

// kPer: consecutive tokens of a thread; kCtas: of a cluster
template <int D, int kThreads, int kPer, int kCtas>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 4 : kThreads == 512 ? 2 : 1) kv_evict_kernel(const Args a) {
  constexpr int kWarps = kThreads / 32, kStep = kThreads * kPer;
  __shared__ uint32_t hist[2][kBins];  // two digits' in turn: a CTA may still read the last one's
  __shared__ uint32_t s_warp[2][kWarps], s_pick[2], s_total[2];
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
  for (int i = keep + rank * kThreads + tid; i < a.budget; i += kCtas * kThreads) kept[i] = -1;
  for (int i = keep + rank * kThreads + tid; i < a.new_cap; i += kCtas * kThreads) nw[i] = 0.f;
  const int rounds = (n + kCtas * kStep - 1) / (kCtas * kStep);  // 1: all tokens are in registers
  // the tokens of a round: thread by thread, CTA by CTA; a row of weights begins at a 16-byte boundary (cap is a multiple of 16)
  float x[kPer];
  auto load = [&](int round) {
    const int t0 = ((round * kCtas + rank) * kThreads + tid) * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const float4 v = t0 + i < n ? *reinterpret_cast<const float4*>(w + t0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
    return t0;
  };
  int t0 = load(0);
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
        // a run of equal digits is counted once
        uint32_t last = 0xffffffffu, cnt = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t k = order_of(x[i]);
          if (t0 + i >= old || (k & mask) != prefix) continue;
          const uint32_t bin = k >> shift & (bins - 1);
          if (bin != last) {
            if (cnt) atomicAdd(&h[last], cnt);
            last = bin, cnt = 0;
          }
          ++cnt;
        }
        if (cnt) atomicAdd(&h[last], cnt);
      }
      sync_all();
      // the bin that holds the last kept one, counting from the greatest: a thread's bins, all CTAs' counts
      constexpr int kEach = kBins / kThreads;
      uint32_t c[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int bin = bins - 1 - (tid * kEach + i);
        c[i] = 0;
        if (bin >= 0) {
          if (kCtas == 1) {
            c[i] = h[bin];
          } else {
#pragma unroll
            for (int p = 0; p < kCtas; ++p) c[i] += ld_peer(&h[bin], p);
          }
        }
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
          if (above < need && need <= above + c[i]) s_pick[0] = bins - 1 - (tid * kEach + i), s_pick[1] = need - above;
          above += c[i];
        }
      }
      __syncthreads();
      prefix |= s_pick[0] << shift;
      need = s_pick[1];
    }
    ties = need;
  }
  // counting off: tokens before this thread's that are greater than the smallest kept number or too new to compete, and ties
  uint32_t done = 0, met = 0;  // of the rounds before
  for (int r = 0; r < rounds; ++r) {
    if (rounds > 1) t0 = load(r);
    uint32_t sure = 0, tie = 0;  // bits
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t k = order_of(x[i]);
      const bool comp = t0 + i < old;
      if (t0 + i < n && (!comp || (search ? k > prefix : places > 0))) sure |= 1u << i;
      if (search && comp && k == prefix) tie |= 1u << i;
    }
    uint32_t both = __popc(sure) | __popc(tie) << 16, incl = both;  // a CTA has 2^14 tokens at most
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += o;
    }
    __syncthreads();
    if (lane == 31) s_warp[r & 1][warp] = incl;
    __syncthreads();
    uint32_t total = 0;
    for (int v = 0; v < kWarps; ++v) {
      if (v < warp) incl += s_warp[r & 1][v];
      total += s_warp[r & 1][v];
    }
    uint32_t at = done + ((incl - both) & 0xffffu), ties_at = met + ((incl - both) >> 16);
    if (kCtas > 1) {
      if (tid == 0) s_total[r & 1] = total;
      cluster_sync();
#pragma unroll
      for (int p = 0; p < kCtas; ++p) {
        const uint32_t v = ld_peer(&s_total[r & 1], p);
        if (p < rank) at += v & 0xffffu, ties_at += v >> 16;
        done += v & 0xffffu, met += v >> 16;
      }
    } else {
      done += total & 0xffffu, met += total >> 16;
    }
    // of the ties before this thread, as many are kept as there is room for
    at += min(ties_at, ties);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      bool in = sure >> i & 1;
      if (tie >> i & 1) in = ties_at++ < ties;
      if (in) kept[at] = t0 + i, nw[at] = x[i], ++at;
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

// Tokens as the table's width allows for decide how many threads a head gets, so that they fit the registers.  Many heads get
// smaller clusters, which read longer contexts again for each digit, rather than wait for room.
template <int D>
cudaError_t launch(const Args& a, cudaStream_t s) {
  const long long heads = (long long)a.B * a.H, sms = num_sms();
  if (a.cap <= 1024) return launch<D, 256, 4, 1>(a, s);
  if (a.cap <= 4096) return launch<D, 256, 16, 1>(a, s);
  if (a.cap <= 16384 || heads * 8 > 4 * sms) return launch<D, 512, 16, 2>(a, s);
  if (a.cap <= 65536) return launch<D, 512, 16, 8>(a, s);
  return launch<D, 1024, 16, 8>(a, s);
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
