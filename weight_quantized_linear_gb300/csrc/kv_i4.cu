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

// Every CTA scans the requests' lengths itself (new tokens and new pages of at most kPlanPer requests per thread, all
// loaded before any is used) and then fills its own slots, so that nothing has to be passed between CTAs and one launch
// does it all.  The table entries read here (pages held already) and those written (new pages) are different ones.
// Latency is what it takes: a launch, the loads of the lengths, two barriers, and the loads of a page number (8 requests
// 4.3 us, 256 with 97005 new tokens 4.9 us, 4096 requests 11.5 to 12.8 us).
constexpr int kPlanPer = kPlanMaxB / kPlanThreads;

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(
    const int* __restrict__ ctx_lens, const int* __restrict__ new_lens, int B, int ps, FastDiv by_ps,
    const int* __restrict__ free_pages, int free_cap, const int* __restrict__ free_count, int* table, int width, int T,
    int* __restrict__ cu_new, int* __restrict__ kv_lens, int* __restrict__ slots, int* __restrict__ free_count_out) {
  __shared__ int cu[kPlanMaxB + 1];   // first new token of each request
  __shared__ int off[kPlanMaxB + 1];  // new pages of the requests before it; -1: refused
  __shared__ long long sum_t[kPlanThreads / 32], sum_p[kPlanThreads / 32];
  __shared__ int taken[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  grid_dependency_wait();  // the lengths may come from the preceding kernel
  grid_dependents_launch();
  const int nfree = min(max(free_count[0], 0), free_cap);
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, B), cnt = min(per, B - r0);
  auto pages = [&](int n) {  // ceil(n / ps)
    const int q = (int)quot((uint32_t)n, by_ps);
    return q + (q * ps != n);
  };
  int c[kPlanPer], n[kPlanPer], need[kPlanPer];  // need: pages beyond those held; -1 if the table row is too short
  long long tok = 0, pg = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    c[k] = k < cnt ? max(ctx_lens[r0 + k], 0) : 0;
    n[k] = k < cnt ? max(new_lens[r0 + k], 0) : 0;
  }
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const long long most = (long long)width * ps;  // below 2^31
    need[k] = (long long)c[k] + n[k] > most ? -1 : pages(c[k] + n[k]) - pages(c[k]);
    tok += n[k];
    pg += max(need[k], 0);
  }
  long long t = tok, p = pg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ot = __shfl_up_sync(0xffffffffu, t, d), op = __shfl_up_sync(0xffffffffu, p, d);
    if (lane >= d) t += ot, p += op;
  }
  if (lane == 31) sum_t[wid] = t, sum_p[wid] = p;
  __syncthreads();
  for (int w = 0; w < wid; ++w) t += sum_t[w], p += sum_p[w];
  t -= tok, p -= pg;
  int used = 0;  // those who are served take a run of the list from its end: its length is the furthest one's
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    if (k >= cnt) break;
    const int r = r0 + k;
    const bool ok = need[k] == 0 || (need[k] > 0 && p + need[k] <= nfree);
    cu[r] = (int)min(t, (long long)INT_MAX);
    off[r] = ok ? (int)min(p, (long long)INT_MAX) : -1;
    if (blockIdx.x == 0) {
      cu_new[r] = cu[r];
      kv_lens[r] = ok ? c[k] + n[k] : 0;
    }
    if (ok && need[k] > 0) used = (int)p + need[k];
    t += n[k];
    p += max(need[k], 0);
  }
  if (tid == 0 && B == 0) cu[0] = 0;
  if (r0 < B && r0 + cnt == B) cu[B] = (int)min(t, (long long)INT_MAX);
  used = __reduce_max_sync(0xffffffffu, used);
  if (lane == 0) taken[wid] = used;
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    for (int w = 1; w < kPlanThreads / 32; ++w) used = max(used, taken[w]);
    *free_count_out = nfree - used;
    cu_new[B] = cu[B];
  }

  // the requests' new pages: a warp per request
  for (int r = blockIdx.x * (kPlanThreads / 32) + wid; r < B; r += gridDim.x * (kPlanThreads / 32)) {
    if (off[r] < 0) continue;
    const int len = max(ctx_lens[r], 0), held = pages(len), more = pages(len + max(new_lens[r], 0)) - held;
    for (int k = lane; k < more; k += 32) table[(size_t)r * width + held + k] = free_pages[nfree - 1 - off[r] - k];
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
      const int len = max(ctx_lens[lo], 0);
      const int pos = len + (tt - cu[lo]), k = (int)quot((uint32_t)pos, by_ps), held = pages(len);
      const int page = k < held ? table[(size_t)lo * width + k] : free_pages[nfree - 1 - off[lo] - (k - held)];
      const long long slot = (long long)page * ps + (pos - k * ps);
      if (page >= 0 && slot <= INT_MAX) out[j] = (int)slot;
    }
  }
  if (t0 <= T - 4) {
    *reinterpret_cast<int4*>(slots + t0) = make_int4(out[0], out[1], out[2], out[3]);
  } else {
    for (int j = 0; j < T - t0; ++j) slots[t0 + j] = out[j];
  }
}

// ---------------------------------------------------------------------------------------------
// Quantise and append
// ---------------------------------------------------------------------------------------------

constexpr int kAppendThreads = 128;

// The exact remainder of d = fl(x - y): x - y = d + remainder (Knuth's two-sum of x and -y).
__device__ __forceinline__ float kv_rest(float x, float y, float d) {
  const float b = __fsub_rn(d, x);
  return __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-y, b));
}

// fp16((max - lo) / 15) of the real quotient, from d = fl(max - lo) and its remainder e.  fl(d * fl(1 / 15)) is within 2 fp32 ulps of the real quotient, so only when it comes within 4 ulps
// of the middle between two fp16 numbers can its rounding differ from the real quotient's; there the sign of
// (d - 15 tie) + e decides, whose first difference is exact (both are close, 15 tie has 16 bits).  Below
// 2^-14 (fp16 subnormals) x is a small multiple of 2^-24, d is exact, and n / 15 is never a tie.
__device__ __forceinline__ __half kv_scale(float hi, float lo, float d) {
  const float q = __fmul_rn(d, 1.0f / 15.0f);
  const unsigned b = __float_as_uint(q), low = b & 0x1fffu;
  float r = q;
  if (q >= 6.103515625e-05f && low - 0xffcu <= 8u) {
    const float tie = __uint_as_float((b & ~0x1fffu) | 0x1000u);
    const float s = __fadd_rn(__fsub_rn(d, __fmul_rn(15.0f, tie)), kv_rest(hi, lo, d));
    r = s > 0.f ? __uint_as_float(__float_as_uint(tie) + 1) : s < 0.f ? __uint_as_float(__float_as_uint(tie) - 1) : tie;
  }
  const __half h = __float2half_rn(r);
  return __half_as_ushort(h) == 0 ? __ushort_as_half(0x3c00) : h;
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 kv_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 kv_add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// round_half_even((x - lo) / s) of the real quotient, where fl(x - lo) * fl(1 / s) comes within 1e-5 of the middle
// between c and c + 1: the sign of ((x - lo) - (c + 1/2) s) decides, computed exactly: x - lo = d + e, (c + 1/2) s has
// 16 bits, and d minus it is exact because the two are close.
__device__ __forceinline__ float kv_code_near_tie(float x, float lo, float s, float inv) {
  const float d = __fsub_rn(x, lo), fl = floorf(__fmul_rn(d, inv));
  const float r = __fadd_rn(__fsub_rn(d, __fmul_rn(fl + 0.5f, s)), kv_rest(x, lo, d));
  return fl + (r > 0.f || (r == 0.f && ((int)fl & 1)) ? 1.0f : 0.0f);
}

// The codes clamp(round_half_even((x - lo) / s), 0, 15) of eight values, the first in the lowest bits.
// y = fl(d * inv + 1.5 * 2^23) with d = fl(x - lo), inv within 2^-23 of 1 / s is that magic number plus the integer nearest
// to d * inv, which is off the quotient by at most 2^-22 * 16 < 4e-6, so that integer is the code unless the rest
// d * inv - integer (exact up to one rounding) comes within 1e-5 of a half; then kv_code_near_tie decides.  x >= lo, and
// d * inv <= 15.01 unless s has lost bits below 2^-14, where the codes are clamped.  Four codes are added up, times powers
// of 16, in fp32 (below 2^16 and exact); their sum stands in the low bits of 2^23 plus it.  Ties are not rare (differences
// and scales have 11 bits): one lane in a hundred has one, one warp in four, so they are taken one at a time.
__device__ __forceinline__ uint32_t kv_codes(const uint4& raw, float lo, float s, float inv) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
  const float2 nlo = make_float2(-lo, -lo), i2 = make_float2(inv, inv), mg = make_float2(kMagic, kMagic),
               minus = make_float2(-1.f, -1.f);
  float2 f[4], n[4];  // what rounding left, minus the codes
  float rest = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = kv_add2(__half22float2(*reinterpret_cast<const __half2*>(&r[j])), nlo);
    n[j] = kv_fma2(kv_fma2(d, i2, mg), minus, mg);
    f[j] = kv_fma2(d, i2, n[j]);
    asm("max.f32 %0, %0, %1, %2;" : "+f"(rest) : "f"(fabsf(f[j].x)), "f"(fabsf(f[j].y)));
  }
  if (s < 6.103515625e-05f) {  // 2^-14
#pragma unroll
    for (int j = 0; j < 4; ++j) n[j] = make_float2(fmaxf(n[j].x, -15.f), fmaxf(n[j].y, -15.f));
  }
  const float2 p256 = make_float2(256.f, 256.f), a = kv_fma2(n[1], p256, n[0]), b = kv_fma2(n[3], p256, n[2]);
  const uint32_t low = __float_as_uint(fmaf(a.y, -16.f, 8388608.f - a.x)), high = __float_as_uint(fmaf(b.y, -16.f, 8388608.f - b.x));
  uint32_t word = __byte_perm(low, high, 0x5410);
  if (rest > 0.49999f) {
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) hits |= (fabsf(f[j].x) > 0.49999f ? 1u << (2 * j) : 0u) | (fabsf(f[j].y) > 0.49999f ? 2u << (2 * j) : 0u);
    do {
      const int k = __ffs(hits) - 1;
      const uint32_t pair = k & 4 ? (k & 2 ? r[3] : r[2]) : (k & 2 ? r[1] : r[0]);
      const float x = __half2float(__ushort_as_half((unsigned short)(k & 1 ? pair >> 16 : pair)));
      const uint32_t code = min((int)kv_code_near_tie(x, lo, s, inv), 15);
      word = (word & ~(15u << (4 * k))) | (code << (4 * k));
      hits &= hits - 1;
    } while (hits);
  }
  return word;
}

// A warp takes kTokens consecutive tokens of one head, of K or of V; a row is held by four lanes, each with D / 32 chunks
// of 8 channels (one 16-byte load, one 4-byte store of codes).  More lanes per row spend more on the row's minimum,
// maximum and scale, which all its lanes work out: 8190 tokens of 32 heads of 128 take 42.4 us with 16 lanes, 33.7 with
// 8, 28.1 with 4, 30.9 with 2; 27.3 in blocks of four warps instead of eight (170 MB, 6.2 TB/s, what reading back takes).
template <int D, int kTokens>
__global__ void __launch_bounds__(kAppendThreads) kv_append_i4_kernel(
    const __half* __restrict__ k, const __half* __restrict__ v, long long k_stride, long long v_stride, int T, int H,
    const int* __restrict__ slots, uint8_t* __restrict__ cache, int pages, int ps, FastDiv by_ps, FastDiv by_h,
    unsigned* err) {
  using L = KvI4<D>;
  constexpr int kLanes = 4, kChunks = D / (8 * kLanes), kRows = 32 / kLanes, kIter = kTokens / kRows;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, rl = lane / kLanes;
  grid_dependency_wait();  // k and v may come from the preceding kernel
  grid_dependents_launch();
  const uint32_t unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);  // (tokens, head, K or V)
  const uint32_t tb = quot(unit >> 1, by_h);
  const int is_v = (int)(unit & 1), h = (int)((unit >> 1) - tb * H);
  const long long t0 = (long long)tb * kTokens;
  if (t0 >= T) return;
  const __half* src = is_v ? v : k;
  const long long stride = is_v ? v_stride : k_stride;
  uint4 raw[kIter][kChunks];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const long long t = t0 + i * kRows + rl;
#pragma unroll
    for (int m = 0; m < kChunks; ++m)
      raw[i][m] = t < T ? __ldcs(reinterpret_cast<const uint4*>(src + t * stride + (long long)h * D) + sub + m * kLanes)
                        : make_uint4(0u, 0u, 0u, 0u);
  }
  // lane t % kTokens: where token t goes, its block's offset (a multiple of 128) plus its row there; -1: nowhere
  long long to = -1;
  if (const long long t = t0 + lane % kTokens; t < T) {
    if (const int slot = __ldg(slots + t); slot >= 0) {
      const int page = (int)quot((uint32_t)slot, by_ps), at = slot - page * ps;
      if (page < pages)
        to = (((long long)page * H + h) * (ps / kKvBlock) + at / kKvBlock) * L::kBytes + at % kKvBlock;
      else if (lane < kTokens)
        report_error(err, kErrBadIndex);
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    // the row's minimum and maximum, NaN if it holds one: (min, -max) travel as one pair
    __half2 a, b;
#pragma unroll
    for (int m = 0; m < kChunks; ++m) {
      const __half2* x2 = reinterpret_cast<const __half2*>(&raw[i][m]);
      const __half2 a1 = __hmin2_nan(__hmin2_nan(x2[0], x2[1]), __hmin2_nan(x2[2], x2[3]));
      const __half2 b1 = __hmax2_nan(__hmax2_nan(x2[0], x2[1]), __hmax2_nan(x2[2], x2[3]));
      a = m ? __hmin2_nan(a, a1) : a1, b = m ? __hmax2_nan(b, b1) : b1;
    }
    __half2 mm = __halves2half2(__hmin_nan(__low2half(a), __high2half(a)), __hneg(__hmax_nan(__low2half(b), __high2half(b))));
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float lo = __low2float(mm), hi = -__high2float(mm);
    const float d = __fsub_rn(hi, lo);
    const __half sh = kv_scale(hi, lo, d);
    const float s = __half2float(sh);
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    uint32_t word[kChunks];
#pragma unroll
    for (int m = 0; m < kChunks; ++m) word[m] = kv_codes(raw[i][m], lo, s, inv);
    uint32_t par = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(__low2half(mm)) << 16);
    if (!(d <= 131008.f)) {  // some value is not finite
      par = 0x7fff7fffu;
#pragma unroll
      for (int m = 0; m < kChunks; ++m) word[m] = 0;
    }
    const long long dst = __shfl_sync(0xffffffffu, to, i * kRows + rl);
    if (dst < 0) continue;
    const int row = (int)dst & (kKvBlock - 1);
    uint8_t* blk = cache + (dst - row);
#pragma unroll
    for (int m = 0; m < kChunks; ++m)
      *reinterpret_cast<uint32_t*>(blk + (is_v ? L::kV : 0) + row * L::kRow + 4 * (sub + m * kLanes)) = word[m];
    if (sub == 0) *reinterpret_cast<uint32_t*>(blk + (is_v ? L::kVp : L::kKp) + 4 * row) = par;
  }
}

// ---------------------------------------------------------------------------------------------
// Read back
// ---------------------------------------------------------------------------------------------

constexpr int kReadThreads = 256;

// A thread reads 8 channels (4 bytes of codes) of one row of K and of V and writes 16 bytes to each output; rows of
// negative slots read as zeros.  A stream: 8190 tokens of 32 heads of 128 take 27 us (170 MB, 6.3 TB/s).
template <int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_i4_kernel(const uint8_t* cache, int pages, int ps, FastDiv by_ps,
                                                                  int H, FastDiv by_h, const int* __restrict__ slots, int T,
                                                                  __half* __restrict__ k, __half* __restrict__ v,
                                                                  unsigned* err) {
  using L = KvI4<D>;
  constexpr int kLanes = D / 8;
  const long long n = (long long)T * H * kLanes;
  const int bpp = ps / kKvBlock;
  grid_dependency_wait();  // the cache may come from the preceding kernel
  grid_dependents_launch();
  for (long long i = (long long)blockIdx.x * kReadThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kReadThreads) {
    const int sub = (int)(i % kLanes);
    const uint32_t th = (uint32_t)(i / kLanes), t = quot(th, by_h);  // T * H is below 2^31
    const int h = (int)(th - t * H), slot = __ldg(slots + t);
    __align__(16) __half2 o[2][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j >> 2][j & 3] = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
    const int page = slot < 0 ? -1 : (int)quot((uint32_t)slot, by_ps), at = slot - page * ps;
    if (slot >= 0 && page >= pages) report_error(err, kErrBadIndex);
    if (slot >= 0 && page < pages) {
      const uint8_t* blk = cache + (((long long)page * H + h) * bpp + at / kKvBlock) * L::kBytes;
      const int row = at % kKvBlock;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + (s ? L::kV : 0) + row * L::kRow + 4 * sub);
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
    const long long at8 = (long long)th * kLanes + sub;
    __stcs(reinterpret_cast<uint4*>(k) + at8, *reinterpret_cast<const uint4*>(o[0]));
    __stcs(reinterpret_cast<uint4*>(v) + at8, *reinterpret_cast<const uint4*>(o[1]));
  }
}

// A launch that may start before the kernel ahead of it has ended; the kernels wait for it before they read anything.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), int grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

cudaError_t launch_kv_plan(const int* ctx_lens, const int* new_lens, int B, int ps, const int* free_pages, int free_cap,
                           const int* free_count, int* table, int width, int T, int* cu_new, int* kv_lens, int* slots,
                           int* free_count_out, cudaStream_t s) {
  // a CTA for every kPlanSlots slots, and enough for four requests' tables per warp
  const int for_slots = (int)(((long long)T + kPlanSlots - 1) / kPlanSlots), for_pages = (B + 31) / 32;
  const int grid = for_slots > for_pages ? for_slots : for_pages > 0 ? for_pages : 1;
  return launch_early(kv_plan_kernel, grid, kPlanThreads, s, ctx_lens, new_lens, B, ps, fast_div(ps), free_pages, free_cap,
                      free_count, table, width, T, cu_new, kv_lens, slots, free_count_out);
}

cudaError_t launch_kv_append_i4(const uint16_t* k, const uint16_t* v, long long k_stride, long long v_stride, int T,
                                int H, int D, const int* slots, uint8_t* cache, long long pages, int ps,
                                unsigned* dev_err, cudaStream_t s) {
  // 16 tokens per warp where that still gives every SM 40 warps (of 64 that fit), else 8: 4099 tokens of 8 heads of 64
  // (27 warps of 16) take 3.7 us with 8 and 4.4 with 16, 8190 of them (54) 6.1 and 5.7, 8190 of 32 heads of 128 30.3 and 27.8
  const long long warps = ((long long)T + 15) / 16 * 2 * H, per = kAppendThreads / 32;
  const bool many = warps >= 40LL * num_sms();
  const long long units = many ? warps : ((long long)T + 7) / 8 * 2 * H, grid = (units + per - 1) / per;
  auto* kernel = D == 128 ? (many ? kv_append_i4_kernel<128, 16> : kv_append_i4_kernel<128, 8>)
                          : (many ? kv_append_i4_kernel<64, 16> : kv_append_i4_kernel<64, 8>);
  return launch_early(kernel, (int)grid, kAppendThreads, s, reinterpret_cast<const __half*>(k),
                      reinterpret_cast<const __half*>(v), k_stride, v_stride, T, H, slots, cache, (int)pages, ps,
                      fast_div(ps), fast_div(H), dev_err);
}

cudaError_t launch_kv_read_i4(const uint8_t* cache, long long pages, int ps, int H, int D, const int* slots, int T,
                              uint16_t* k, uint16_t* v, unsigned* dev_err, cudaStream_t s) {
  const long long n = (long long)T * H * (D / 8), want = (n + kReadThreads - 1) / kReadThreads;
  const long long cap = 8LL * num_sms();
  auto* kernel = D == 128 ? kv_read_i4_kernel<128> : kv_read_i4_kernel<64>;
  return launch_early(kernel, (int)(want < cap ? want : cap), kReadThreads, s, cache, (int)pages, ps, fast_div(ps), H, fast_div(H),
                      slots, T, reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v), dev_err);
}

}  // namespace wql
