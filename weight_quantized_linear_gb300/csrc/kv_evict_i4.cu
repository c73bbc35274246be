// kv_evict_i4.cu -- leaving the least attended tokens of a paged 4-bit KV cache behind.
//
// Of the n = kv_lens[b] tokens of sequence b, each K/V head keeps min(n, budget): the last min(recent, budget) ones and, of
// the others, those with the greatest weights (of equal ones the first; a NaN counts as greater than any number).  The kept
// ones go, in their order, into the pages of row b of new_table; their numbers and weights go to kept and new_weights.
//
// The selection finds the smallest kept weight, digit by digit of a 32-bit number that orders as the weights do, and then
// counts off the kept tokens in their order.  The rows are moved by a second kernel, a warp per block of 16.
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kSelThreads = 1024, kMoveThreads = 256;

struct Args {
  const float* weights;  // [B, H, cap]
  uint8_t* cache;
  int pages, ps, H;
  FastDiv by_ps;
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

__global__ void __launch_bounds__(kSelThreads) kv_evict_select_kernel(const Args a) {
  __shared__ unsigned hist[256], warp_sum[kSelThreads / 32], s_prefix, s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.x / a.H;
  int n = max(a.kv_lens[b], 0);
  if (n > a.cap) {
    if (tid == 0) report_error(a.err, kErrBadIndex);
    n = a.cap;
  }
  const int keep = min(n, a.budget), old = n - min(min(a.recent, a.budget), n);  // tokens 0 .. old - 1 compete
  const float* w = a.weights + (long long)blockIdx.x * a.cap;
  int* kept = a.kept + (long long)blockIdx.x * a.budget;
  float* nw = a.new_weights + (long long)blockIdx.x * a.new_cap;
  if (blockIdx.x % a.H == 0 && tid == 0) a.new_lens[b] = keep;
  const int places = keep - (n - old);  // of the competing ones are kept
  uint32_t prefix = 0;                  // the smallest kept weight's number
  unsigned ties = 0;                    // and how many of those that have it
  if (places < old && places > 0) {
    unsigned need = places;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
      for (int t = tid; t < old; t += kSelThreads) {
        const uint32_t k = order_of(w[t]);
        if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        unsigned above = 0;
        while (above + hist[d] < need) above += hist[d--];
        s_prefix = prefix | (uint32_t)d << shift;
        s_need = need - above;
      }
      __syncthreads();
      prefix = s_prefix, need = s_need;
    }
    ties = need;
  }
  const bool all = places >= old, none = places == 0;
  unsigned done = 0, met = 0;  // kept so far, ties met so far
  for (int t0 = 0; t0 < n; t0 += kSelThreads) {
    const int t = t0 + tid;
    const float x = t < n ? w[t] : 0.f;
    const uint32_t k = order_of(x);
    const bool comp = t < old, tie = comp && !all && !none && k == prefix;
    bool in = t < n && (!comp || all || (!none && k > prefix));
    // among the ties, the first ones
    const unsigned tb = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) warp_sum[warp] = __popc(tb);
    __syncthreads();
    unsigned before = met, sum = 0;
    for (int v = 0; v < kSelThreads / 32; ++v) {
      if (v < warp) before += warp_sum[v];
      sum += warp_sum[v];
    }
    met += sum;
    if (tie) in = before + __popc(tb & ((1u << lane) - 1)) < ties;
    __syncthreads();
    const unsigned ib = __ballot_sync(0xffffffffu, in);
    if (lane == 0) warp_sum[warp] = __popc(ib);
    __syncthreads();
    unsigned at = done;
    sum = 0;
    for (int v = 0; v < kSelThreads / 32; ++v) {
      if (v < warp) at += warp_sum[v];
      sum += warp_sum[v];
    }
    done += sum;
    at += __popc(ib & ((1u << lane) - 1));
    if (in) kept[at] = t, nw[at] = x;
    __syncthreads();
  }
  for (int i = keep + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  for (int i = keep + tid; i < a.new_cap; i += kSelThreads) nw[i] = 0.f;
}

// A warp moves the rows of one block of 16 tokens of a K/V head: 16 bytes of codes per lane at a time.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(const Args a) {
  using L = KvI4<D>;
  constexpr int kChunks = 2 * L::kRow / 16;  // of 16 bytes, per token: K's, then V's
  const int lane = threadIdx.x & 31;
  const int per = (a.budget + kKvBlock - 1) / kKvBlock, bpp = a.ps / kKvBlock;
  grid_dependency_wait();
  grid_dependents_launch();
  const long long units = (long long)a.B * a.H * per;
  for (long long u = (long long)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); u < units;
       u += (long long)gridDim.x * (kMoveThreads / 32)) {
    const int blk = (int)(u % per);
    const long long bh = u / per;
    const int b = (int)(bh / a.H), h = (int)(bh % a.H);
    const int cnt = min(min(max(a.kv_lens[b], 0), min(a.cap, a.budget)) - blk * kKvBlock, kKvBlock);
    if (cnt <= 0) continue;
    const int to = a.new_table[(long long)b * a.new_width + blk / bpp];
    if (to < 0 || to >= a.pages) {
      report_error(a.err, kErrBadIndex);
      continue;
    }
    uint8_t* dst = a.cache + (((long long)to * a.H + h) * bpp + blk % bpp) * L::kBytes;
    long long from = -1;  // lane: where token lane % 16 is, its block's offset (a multiple of 128) plus its row there
    if ((lane & 15) < cnt) {
      const int t = a.kept[bh * a.budget + blk * kKvBlock + (lane & 15)];
      const int pg = (int)quot((uint32_t)t, a.by_ps), at = t - pg * a.ps, page = a.table[(long long)b * a.width + pg];
      if (page < 0 || page >= a.pages)
        report_error(a.err, kErrBadIndex);
      else
        from = (((long long)page * a.H + h) * bpp + at / kKvBlock) * L::kBytes + at % kKvBlock;
    }
#pragma unroll
    for (int i = 0; i < kKvBlock * kChunks / 32; ++i) {
      const int row = (i * 32 + lane) / kChunks, ch = (i * 32 + lane) % kChunks;
      const long long f = __shfl_sync(0xffffffffu, from, row);
      if (f < 0) continue;
      const int r = (int)f & (kKvBlock - 1), part = ch >= kChunks / 2 ? L::kV : 0, c = ch % (kChunks / 2);
      *reinterpret_cast<uint4*>(dst + part + row * L::kRow + 16 * c) =
          *reinterpret_cast<const uint4*>(a.cache + (f - r) + part + r * L::kRow + 16 * c);
    }
    if (from >= 0) {  // lanes 0-15: K's parameters, 16-31: V's
      const int r = (int)from & (kKvBlock - 1), part = lane < 16 ? L::kKp : L::kVp;
      *reinterpret_cast<uint32_t*>(dst + part + 4 * (lane & 15)) =
          *reinterpret_cast<const uint32_t*>(a.cache + (from - r) + part + 4 * r);
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict_i4(const float* weights, uint8_t* cache, long long pages, int ps, int H, int D, const int* table,
                               int width, const int* kv_lens, int B, const int* new_table, int new_width, int budget,
                               int recent, int* kept, float* new_weights, int* new_lens, unsigned* dev_err, cudaStream_t s) {
  Args a{weights, cache, (int)pages, ps, H, fast_div(ps), table, width, width * ps, kv_lens, B, new_table, new_width,
         new_width * ps, budget, recent, kept, new_weights, new_lens, dev_err};
  kv_evict_select_kernel<<<B * H, kSelThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long warps = (long long)B * H * ((budget + kKvBlock - 1) / kKvBlock), per = kMoveThreads / 32;
  const long long want = (warps + per - 1) / per, cap = 16LL * num_sms();
  const int grid = (int)(want < cap ? want : cap);
  if (D == 128)
    kv_evict_move_kernel<128><<<grid, kMoveThreads, 0, s>>>(a);
  else
    kv_evict_move_kernel<64><<<grid, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace wql
