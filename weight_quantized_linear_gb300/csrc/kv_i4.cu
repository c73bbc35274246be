// kv_i4.cu -- the paged 4-bit KV cache: page planning from request lengths, quantising new K and V rows
// into it, and reading rows back.
//
// A row is one token's K or V vector of one head, x [D] fp16.  With lo = min x and s =
// fp16((max x - lo) / 15) (1.0 if that is zero), code = clamp(round_half_even((x - lo) / s), 0, 15) and
// the value read back is fp16(code * s + lo).  The quotients are the real ones: every code and scale is
// what exact arithmetic rounded once gives, so that any implementation of the definition agrees bit for
// bit.  A row that holds an infinity or a NaN is stored with s = lo = NaN: it reads back as NaN.
#include <climits>

#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

// ---------------------------------------------------------------------------------------------
// Page planning
// ---------------------------------------------------------------------------------------------

constexpr int kPlanThreads = 256;
constexpr int kPlanSlots = 4 * kPlanThreads;  // slots per CTA

// Inclusive scan over the CTA of one 64-bit value per thread.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // warp_sums may still be read from the scan before
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += warp_sums[w];
  return v;
}

// Every CTA scans the requests' lengths itself (two values per request, at most 16 requests per thread)
// and then fills its own slots, so that nothing has to be passed between CTAs and one launch does it all.
// The table entries read here (pages held already) and those written (new pages) are different ones.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(
    const int* __restrict__ ctx_lens, const int* __restrict__ new_lens, int B, int ps, const int* __restrict__ free_pages,
    int free_cap, const int* __restrict__ free_count, int* table, int width, int T, int* __restrict__ cu_new,
    int* __restrict__ kv_lens, int* __restrict__ slots, int* __restrict__ free_count_out) {
  __shared__ int cu[kPlanMaxB + 1];   // first new token of each request
  __shared__ int off[kPlanMaxB + 1];  // new pages of the requests before it; -1: refused
  __shared__ long long sums[kPlanThreads / 32];
  const int tid = threadIdx.x;
  const int nfree = min(max(free_count[0], 0), free_cap);
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
  // pages a request needs beyond those it holds; -1 if its table row is too short
  auto pages_of = [&](int c, int n) -> long long {
    const long long total = ((long long)c + n + ps - 1) / ps;
    return total > width ? -1 : total - (c + (ps - 1LL)) / ps;
  };
  long long tok = 0, pg = 0;
  for (int r = r0; r < r1; ++r) {
    const int c = max(ctx_lens[r], 0), n = max(new_lens[r], 0);
    tok += n;
    pg += max(pages_of(c, n), 0LL);
  }
  const long long tok_incl = block_scan(tok, sums);
  const long long pg_incl = block_scan(pg, sums);
  long long t = tok_incl - tok, p = pg_incl - pg;
  long long taken = 0;
  for (int r = r0; r < r1; ++r) {
    const int c = max(ctx_lens[r], 0), n = max(new_lens[r], 0);
    const long long need = pages_of(c, n);
    const bool ok = need == 0 || (need > 0 && p + need <= nfree);
    cu[r] = (int)min(t, (long long)INT_MAX);
    off[r] = ok ? (int)min(p, (long long)INT_MAX) : -1;
    if (blockIdx.x == 0) {
      cu_new[r] = cu[r];
      kv_lens[r] = ok ? c + n : 0;
    }
    if (ok) taken += need;
    t += n;
    p += max(need, 0LL);
  }
  if (B == 0 && tid == 0) cu[0] = 0;
  if (r1 == B && r0 < B) cu[B] = (int)min(t, (long long)INT_MAX);
  const long long taken_incl = block_scan(taken, sums);
  if (blockIdx.x == 0 && tid == kPlanThreads - 1) *free_count_out = nfree - (int)taken_incl;
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) cu_new[B] = cu[B];

  // the requests' new pages: a warp per request
  const int lane = tid & 31, warp = blockIdx.x * (kPlanThreads / 32) + (tid >> 5);
  for (int r = warp; r < B; r += gridDim.x * (kPlanThreads / 32)) {
    const int c = max(ctx_lens[r], 0), n = max(new_lens[r], 0);
    if (off[r] < 0) continue;
    const int held = (int)((c + (ps - 1LL)) / ps), need = (int)pages_of(c, n);
    for (int k = lane; k < need; k += 32)
      table[(size_t)r * width + held + k] = free_pages[nfree - 1 - off[r] - k];
  }

  // the slots of tokens t0 .. t0 + 3
  const int t0 = blockIdx.x * kPlanSlots + 4 * tid;
  if (t0 >= T) return;
  int lo = 0, hi = B;  // the request of token t0: the last one with cu <= t0
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    (cu[mid] <= t0 ? lo : hi) = mid;
  }
  int out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int tt = t0 + j;
    while (lo + 1 < B && cu[lo + 1] <= tt) ++lo;
    out[j] = -1;
    if (tt < cu[B] && off[lo] >= 0) {
      const int c = max(ctx_lens[lo], 0);
      const int pos = c + (tt - cu[lo]), k = pos / ps, held = (int)((c + (ps - 1LL)) / ps);
      const int page = k < held ? table[(size_t)lo * width + k] : free_pages[nfree - 1 - off[lo] - (k - held)];
      if (page >= 0) out[j] = page * ps + (pos - k * ps);
    }
  }
  if (t0 + 4 <= T) {
    *reinterpret_cast<int4*>(slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
  } else {
    for (int j = 0; t0 + j < T; ++j) slots[t0 + j] = out[j];
  }
}

// ---------------------------------------------------------------------------------------------
// Quantise and append
// ---------------------------------------------------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;  // tokens per warp, of one head and one of K and V

// fp16((max - lo) / 15) of the real quotient, from d + e = max - lo (d the fp32 difference, e its exact
// remainder).  fl(d / 15) is within 2 fp32 ulps of the real quotient, so only when it comes within 4 ulps
// of the middle between two fp16 numbers can its rounding differ from the real quotient's; there the sign of
// (d - 15 tie) + e decides, whose first difference is exact (both are close, 15 tie has 16 bits).  Below
// 2^-14 (fp16 subnormals) x is a small multiple of 2^-24, d is exact, and n / 15 is never a tie.
__device__ __forceinline__ __half kv_scale(float d, float e) {
  const float q = __fdiv_rn(d, 15.0f);
  const unsigned b = __float_as_uint(q), low = b & 0x1fffu;
  float r = q;
  if (q >= 6.103515625e-05f && low - 0xffcu <= 8u) {
    const float tie = __uint_as_float((b & ~0x1fffu) | 0x1000u);
    const float s = __fadd_rn(__fsub_rn(d, __fmul_rn(15.0f, tie)), e);
    r = s > 0.f ? __uint_as_float(__float_as_uint(tie) + 1) : s < 0.f ? __uint_as_float(__float_as_uint(tie) - 1) : tie;
  }
  const __half h = __float2half_rn(r);
  return __half_as_ushort(h) == 0 ? __ushort_as_half(0x3c00) : h;
}

// clamp(round_half_even((x - lo) / s), 0, 15) of the real quotient.  t = fl(fl(x - lo) * fl(1 / s)) is off by
// at most 3 * 2^-24 * 16 < 3e-6, so it decides unless it is that close to a half; then the sign of
// ((x - lo) - (c + 1/2) s) does, computed exactly: x - lo = d + e, (c + 1/2) s has 16 bits, and d minus it
// is exact because the two are close.
__device__ __forceinline__ int kv_code(float x, float lo, float s, float inv) {
  const float d = __fsub_rn(x, lo);
  const float t = __fmul_rn(d, inv);
  const float rt = rintf(t);
  int c = (int)rt;
  if (fabsf(__fsub_rn(t, rt)) > 0.49999f) {
    const float fl = floorf(t);
    // x - lo = d + e (Knuth's two-sum of x and -lo)
    const float bb = __fsub_rn(d, x);
    const float e = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-lo, bb));
    const float r = __fadd_rn(__fsub_rn(d, __fmul_rn(fl + 0.5f, s)), e);
    c = (int)fl;
    if (r > 0.f || (r == 0.f && (c & 1))) ++c;
  }
  return min(max(c, 0), 15);
}

// A warp takes kAppendTokens consecutive tokens of one head, of K or of V; a row is held by D / 8 lanes, 8
// channels (one 16-byte load) each, and its codes are one 4-byte store per lane.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_i4_kernel(
    const __half* __restrict__ k, const __half* __restrict__ v, long long k_stride, long long v_stride, int T, int H,
    const int* __restrict__ slots, uint8_t* __restrict__ cache, long long pages, int ps, unsigned* err) {
  using L = KvI4<D>;
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kIter = kAppendTokens / kRows;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, rl = lane / kLanes;
  const long long unit = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const long long ntb = (T + kAppendTokens - 1) / kAppendTokens;
  if (unit >= ntb * 2 * H) return;
  const int is_v = (int)(unit & 1), h = (int)((unit >> 1) % H);
  const long long t0 = (unit >> 1) / H * kAppendTokens;
  const __half* src = is_v ? v : k;
  const long long stride = is_v ? v_stride : k_stride;
  const int bpp = ps / kKvBlock;
  uint4 raw[kIter];
  int slot[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long t = t0 + i * kRows + rl;
    slot[i] = t < T ? __ldg(slots + t) : -1;
    raw[i] = t < T ? __ldcs(reinterpret_cast<const uint4*>(src + t * stride + (long long)h * D) + sub)
                   : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const __half2* x2 = reinterpret_cast<const __half2*>(&raw[i]);
    // the row's minimum and maximum, NaN if it holds one: (min, -max) travel as one pair
    const __half2 a = __hmin2_nan(__hmin2_nan(x2[0], x2[1]), __hmin2_nan(x2[2], x2[3]));
    const __half2 b = __hmax2_nan(__hmax2_nan(x2[0], x2[1]), __hmax2_nan(x2[2], x2[3]));
    __half2 mm = __halves2half2(__hmin_nan(__low2half(a), __high2half(a)), __hneg(__hmax_nan(__low2half(b), __high2half(b))));
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float lo = __low2float(mm), hi = -__high2float(mm);
    const float d = __fsub_rn(hi, lo);
    uint32_t word = 0, par = 0x7fff7fffu;
    if (isfinite(lo) && isfinite(hi)) {
      const float bb = __fsub_rn(d, hi);
      const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(d, bb)), __fsub_rn(-lo, bb));
      const __half sh = kv_scale(d, e);
      const float s = __half2float(sh), inv = __fdiv_rn(1.0f, s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        word |= (uint32_t)kv_code(__low2float(x2[j]), lo, s, inv) << (8 * j);
        word |= (uint32_t)kv_code(__high2float(x2[j]), lo, s, inv) << (8 * j + 4);
      }
      par = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(__low2half(mm)) << 16);
    }
    if (slot[i] < 0) continue;
    const int page = slot[i] / ps, at = slot[i] - page * ps;
    if (page >= pages) {
      if (sub == 0) report_error(err, kErrBadIndex);
      continue;
    }
    uint8_t* blk = cache + (((long long)page * H + h) * bpp + at / kKvBlock) * L::kBytes;
    const int row = at % kKvBlock;
    *reinterpret_cast<uint32_t*>(blk + (is_v ? L::kV : 0) + row * L::kRow + 4 * sub) = word;
    if (sub == 0) *reinterpret_cast<uint32_t*>(blk + (is_v ? L::kVp : L::kKp) + 4 * row) = par;
  }
}

// ---------------------------------------------------------------------------------------------
// Read back
// ---------------------------------------------------------------------------------------------

constexpr int kReadThreads = 256;

// A thread reads 8 channels (4 bytes of codes) of one row of K and of V and writes 16 bytes to each output; rows of
// negative slots read as zeros.
template <int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_i4_kernel(const uint8_t* __restrict__ cache, long long pages,
                                                                  int ps, int H, const int* __restrict__ slots, int T,
                                                                  __half* __restrict__ k, __half* __restrict__ v,
                                                                  unsigned* err) {
  using L = KvI4<D>;
  constexpr int kLanes = D / 8;
  const long long n = (long long)T * H * kLanes;
  const int bpp = ps / kKvBlock;
  for (long long i = (long long)blockIdx.x * kReadThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kReadThreads) {
    const int sub = (int)(i % kLanes);
    const long long th = i / kLanes;
    const int h = (int)(th % H), slot = __ldg(slots + th / H);
    __align__(16) __half2 o[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j >> 2][j & 3] = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
    const int page = slot / ps, at = slot - page * ps;
    if (slot >= 0 && page >= pages) report_error(err, kErrBadIndex);
    if (slot >= 0 && page < pages) {
      const uint8_t* blk = cache + (((long long)page * H + h) * bpp + at / kKvBlock) * L::kBytes;
      const int row = at % kKvBlock;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(blk + (s ? L::kV : 0) + row * L::kRow + 4 * sub));
        const __half2 par = *reinterpret_cast<const __half2*>(blk + (s ? L::kVp : L::kKp) + 4 * row);
        const __half2 sc = __low2half2(par), lo = __high2half2(par);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // two codes as the fp16 numbers 1024 + code; one add leaves them exact
          const uint32_t c = ((w >> (8 * j)) & 0xfu) | (((w >> (8 * j + 4)) & 0xfu) << 16) | 0x64006400u;
          const uint32_t f = hadd2_u32(c, 0xE400E400u);
          o[s][j] = __hfma2(*reinterpret_cast<const __half2*>(&f), sc, lo);
        }
      }
    }
    const long long at8 = th * kLanes + sub;
    __stcs(reinterpret_cast<uint4*>(k) + at8, *reinterpret_cast<const uint4*>(o[0]));
    __stcs(reinterpret_cast<uint4*>(v) + at8, *reinterpret_cast<const uint4*>(o[1]));
  }
}

}  // namespace

cudaError_t launch_kv_plan(const int* ctx_lens, const int* new_lens, int B, int ps, const int* free_pages, int free_cap,
                           const int* free_count, int* table, int width, int T, int* cu_new, int* kv_lens, int* slots,
                           int* free_count_out, cudaStream_t s) {
  const int grid = T > 0 ? (T + kPlanSlots - 1) / kPlanSlots : 1;
  kv_plan_kernel<<<grid, kPlanThreads, 0, s>>>(ctx_lens, new_lens, B, ps, free_pages, free_cap, free_count, table, width,
                                               T, cu_new, kv_lens, slots, free_count_out);
  return cudaGetLastError();
}

cudaError_t launch_kv_append_i4(const uint16_t* k, const uint16_t* v, long long k_stride, long long v_stride, int T,
                                int H, int D, const int* slots, uint8_t* cache, long long pages, int ps,
                                unsigned* dev_err, cudaStream_t s) {
  const long long units = (long long)((T + kAppendTokens - 1) / kAppendTokens) * 2 * H;
  const long long per = kAppendThreads / 32, grid = (units + per - 1) / per;
  auto* kernel = D == 128 ? kv_append_i4_kernel<128> : kv_append_i4_kernel<64>;
  kernel<<<(unsigned)grid, kAppendThreads, 0, s>>>(reinterpret_cast<const __half*>(k), reinterpret_cast<const __half*>(v),
                                                   k_stride, v_stride, T, H, slots, cache, pages, ps, dev_err);
  return cudaGetLastError();
}

cudaError_t launch_kv_read_i4(const uint8_t* cache, long long pages, int ps, int H, int D, const int* slots, int T,
                              uint16_t* k, uint16_t* v, unsigned* dev_err, cudaStream_t s) {
  const long long n = (long long)T * H * (D / 8), want = (n + kReadThreads - 1) / kReadThreads;
  const long long cap = 8LL * num_sms();
  auto* kernel = D == 128 ? kv_read_i4_kernel<128> : kv_read_i4_kernel<64>;
  kernel<<<(unsigned)(want < cap ? want : cap), kReadThreads, 0, s>>>(
      cache, pages, ps, H, slots, T, reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v), dev_err);
  return cudaGetLastError();
}

}  // namespace wql
