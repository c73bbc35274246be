// kv_weights_i4.cu -- the attention weight that every cached token gets from packed chunks of rows, added to running sums:
//   weights[b, kvh, t] += sum over the rows r of sequence b that see t, and the query heads h of kvh's group, of
//                         exp(scale q[r, h] . k[t] - lse[r, h]),   k = code * s + lo, rounded to fp16.
//
// The sums run over rows, so a warp keeps 32 keys as the first operand of its products (mma.sync, 16 keys x 8 rows x 16
// channels) in registers, made fp16 there: a lane of the fragment needs two keys' rows, and as the products do not mind the
// order of the channels, it takes 16 contiguous bytes of codes of each.  K is read from memory once and goes nowhere else.
// The rows (token, query head) come in tiles of 64 through shared memory, their channels in the same order; a lane holds two
// keys' scores of two rows, turns them into weights and adds them up in registers.
//
// A unit is 256 keys of a K/V head, a step 64 rows of a unit.  The steps of all units are divided evenly over the CTAs, two
// per SM; sums of units that CTAs share go to the workspace, and a second kernel adds them in their order.
#include <climits>

#include "attn.cuh"
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kPerSm = 2;
constexpr int kUnit = 256, kRows = 64;  // keys of a unit, rows of a step
constexpr int kLead = 1;                // steps that stand for a unit's own cost
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const __half* q;
  long long q_stride;
  int T, Hq, Hkv, G;
  FastDiv by_g;
  const uint8_t* cache;
  int pages, bpp;  // bpp: blocks of a page
  FastDiv by_bpp;
  const int* table;
  int width, cap;
  const int *cu, *kv_lens;
  int B;
  float scale_log2;
  const float* lse;
  float* weights;
  // the workspace: the unit that each CTA began and left unfinished {sequence, K/V head, unit of it, 1}, whether it went on
  // with one (1) and ended it (2), and the sums of both [CTA][0: of the one found begun, 1: of the one begun][kUnit]
  int4* begun;
  int* went_on;
  float* part;
  unsigned* err;
};

// Steps of the units of a sequence: unit u takes the row tiles from skip(u) on, those before see none of its keys.
struct Shape {
  int rows, first, len, units, tiles;
  long long G, c;  // c: row tiles that first tokens fill, rounded up
  __device__ __forceinline__ Shape(const Args& a, const KvChunk& k) : rows(k.rows), first(k.first), len(k.len), G(a.G) {
    units = rows > 0 && len > 0 ? (len - 1) / kUnit + 1 : 0;
    tiles = (int)((rows * G + kRows - 1) / kRows);
    const long long x = first * G;
    c = x >= 0 ? (x + kRows - 1) / kRows : -(-x / kRows);
  }
  static constexpr int kPer = kUnit / kRows;  // row tiles that a unit's keys of one query head fill
  __device__ __forceinline__ int skip(int u) const { return (int)max(kPer * G * u - c, 0LL); }
  __device__ __forceinline__ int cost(int u) const { return kLead + tiles - skip(u); }
  __device__ __forceinline__ long long before(int u) const {  // the cost of units 0 .. u - 1
    const long long u0 = c < 0 ? 0 : min(c / (kPer * G) + 1, (long long)u);  // units that skip nothing
    return (long long)u * (kLead + tiles) - (kPer * G * ((long long)u * (u - 1) - u0 * (u0 - 1)) / 2 - c * (u - u0));
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, kPerSm) kv_weights_i4_kernel(const Args a) {
  using L = KvI4<D>;
  constexpr int kSteps = D / 16;    // products of 16 channels
  constexpr int kWords = D / 32;  // of codes, per lane and key
  __shared__ __align__(16) uint8_t s_q[kRows * D * 2];
  __shared__ __align__(8) float s_lse[kRows];
  __shared__ __align__(8) int s_last[kRows];  // the last key that a row sees
  __shared__ long long s_sum[kWarps], s_off;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
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
    for (int w = 0; w < kWarps; ++w) {
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
  int4 begun = make_int4(0, 0, 0, 0);
  int went_on = 0;
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
    // the codes and parameters of this lane's keys of a unit: keys 16 mt + g and + 8 of the warp's 32
    uint32_t raw[2][2][kWords], par[2][2];
    float old;  // the sum so far of key 16 (c >> 1) + 8 (c & 1) + g
    auto load_keys = [&](int b_, int kvh_, int u_, int len) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const int gb = (u_ * kUnit + 32 * warp) / kKvBlock + mt;
        const bool there = gb * kKvBlock < len;
        const int pg = (int)quot((uint32_t)gb, a.by_bpp), page = there ? a.table[(long long)b_ * a.width + pg] : 0;
        const bool good = there && page >= 0 && page < a.pages;
        if (there && !good) report_error(a.err, kErrBadIndex);
        const uint8_t* blk = a.cache + (((long long)page * a.Hkv + kvh_) * a.bpp + (gb - pg * a.bpp)) * L::kBytes;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = g + 8 * e;
          if constexpr (D == 128) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (good) v = __ldcs(reinterpret_cast<const uint4*>(blk + row * L::kRow) + c);
            raw[mt][e][0] = v.x, raw[mt][e][1] = v.y, raw[mt][e][2] = v.z, raw[mt][e][3] = v.w;
          } else {
            uint2 v = make_uint2(0u, 0u);
            if (good) v = __ldcs(reinterpret_cast<const uint2*>(blk + row * L::kRow) + c);
            raw[mt][e][0] = v.x, raw[mt][e][1] = v.y;
          }
          par[mt][e] = good ? __ldcs(reinterpret_cast<const uint32_t*>(blk + L::kKp) + row) : 0u;
        }
      }
      const int key = u_ * kUnit + 32 * warp + 16 * (c >> 1) + 8 * (c & 1) + g;
      old = key < len ? a.weights[((long long)b_ * a.Hkv + kvh_) * a.cap + key] : 0.f;
    };
    load_keys(b, kvh, u, k.len);
    long long left = w1 - w0;
    int in_b = -1, in_h = -1, in_tile = -1;  // the row tile in shared memory
    while (left > 0) {
      const int skip = sh.skip(u), cost = sh.cost(u), take = (int)min((long long)(cost - s), left);
      const int r0 = max(s - kLead, 0), r1 = s + take - kLead;  // row tiles, from skip on
      // the keys of this unit as fp16 fragments: step s has nibbles 2 (s & 1) and + 1 of word s / 2, with those 4 above them
      uint32_t A[2][kSteps][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t p = kv_finite(par[mt][e]) ? par[mt][e] : 0x7fff7fffu;
          const uint32_t s2 = prmt(p, 0, 0x1010), lo2 = prmt(p, 0, 0x3232);
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            uint32_t h[4];
            kv_values8(raw[mt][e][w], s2, lo2, h);
            if (kv_overflows(p)) {  // rare; of a NaN: no
#pragma unroll
              for (int i = 0; i < 4; ++i) h[i] = kv_clamp2(h[i]);
            }
            A[mt][2 * w][e] = h[0], A[mt][2 * w][2 + e] = h[1];
            A[mt][2 * w + 1][e] = h[2], A[mt][2 * w + 1][2 + e] = h[3];
          }
        }
      const float so_far = old;
      const int key0 = u * kUnit + 32 * warp, ub = b, uh = kvh, uu = u, len = k.len;
      const KvChunk kc = k;
      const int tiles = sh.tiles;
      // the next unit, whose keys are loaded while this one is worked on
      left -= take, s = 0;
      if (left > 0) {
        if (++u == sh.units) {
          u = 0;
          if (++kvh == a.Hkv) {
            kvh = 0;
            do {
              k = kv_chunk(a.cu, a.kv_lens, ++b, a.T, a.cap, nullptr);
              sh = Shape(a, k);
            } while (sh.units == 0);
          }
        }
        load_keys(b, kvh, u, k.len);
      }
      if (r1 <= r0) continue;
      const int slot = r0 > 0 ? 0 : r1 + kLead < cost ? 1 : -1;
      if (slot == 0) went_on = r1 + kLead == cost ? 2 : 1;
      if (slot == 1) begun = make_int4(ub, uh, uu, 1);
      float sum[2][2] = {};
      for (int tile = skip + r0; tile < skip + r1; ++tile) {
        const int i0 = tile * kRows, n = (int)min((long long)kc.rows * a.G - i0, (long long)kRows);
        if (in_b != ub || in_h != uh || in_tile != tile) {
          in_b = ub, in_h = uh, in_tile = tile;
          __syncthreads();  // the tile before is not read any more
          for (int i = tid; i < kRows * (D / 8); i += kThreads) {
            const int row = i / (D / 8), j = i % (D / 8);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < n) {
              const int tok = (int)quot((uint32_t)(i0 + row), a.by_g), h = uh * a.G + (i0 + row - tok * a.G);
              v = *reinterpret_cast<const uint4*>(a.q + (long long)(kc.start + tok) * a.q_stride + (long long)h * D + 8 * j);
            }
            // eight channels as the pairs (0, 4), (1, 5), (2, 6), (3, 7); chunk j is word j % kWords of lane j / kWords
            const int lane_c = j / kWords, w = j % kWords;
            *reinterpret_cast<uint4*>(s_q + row * D * 2 + ((w ^ (row & 1)) * 64 + lane_c * 16)) =
                make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
          }
          if (tid < kRows) {
            float z = INFINITY;  // of a row that does not exist: no weights
            int last = -1;
            if (tid < n) {
              const int tok = (int)quot((uint32_t)(i0 + tid), a.by_g), h = uh * a.G + (i0 + tid - tok * a.G);
              z = a.lse[(long long)(kc.start + tok) * a.Hq + h] * kLog2e;
              last = kc.first + tok;
            }
            s_lse[tid] = z, s_last[tid] = last;
          }
          __syncthreads();
        }
        // whether some row does not see all of the warp's keys
        const bool masked = key0 + 31 > kc.first + (int)quot((uint32_t)i0, a.by_g);
#pragma unroll 1
        for (int nt = 0; nt < (n + 7) / 8; ++nt) {
          float d[2][4] = {};
          const uint32_t src = smem_u32(s_q) + (8 * nt + g) * D * 2 + c * 16;
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            const uint4 bq = lds_u128(src + ((w ^ (g & 1)) * 64));
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              mma_f16_16816(d[mt], A[mt][2 * w], bq.x, bq.y);
              mma_f16_16816(d[mt], A[mt][2 * w + 1], bq.z, bq.w);
            }
          }
          const float2 z = *reinterpret_cast<const float2*>(s_lse + 8 * nt + 2 * c);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float p0 = ex2(fmaf(d[mt][2 * e], a.scale_log2, -z.x)), p1 = ex2(fmaf(d[mt][2 * e + 1], a.scale_log2, -z.y));
              if (masked) {
                const int2 last = *reinterpret_cast<const int2*>(s_last + 8 * nt + 2 * c);
                const int key = key0 + 16 * mt + 8 * e + g;
                if (key > last.x) p0 = 0.f;
                if (key > last.y) p1 = 0.f;
              }
              sum[mt][e] += p0 + p1;
            }
        }
      }
      // over the four lanes that share a key; lane (g, c) then has key 16 (c >> 1) + 8 (c & 1) + g
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[mt][e] += __shfl_xor_sync(0xffffffffu, sum[mt][e], 1);
          sum[mt][e] += __shfl_xor_sync(0xffffffffu, sum[mt][e], 2);
        }
      const float mine = c & 2 ? (c & 1 ? sum[1][1] : sum[1][0]) : (c & 1 ? sum[0][1] : sum[0][0]);
      const int in = 16 * (c >> 1) + 8 * (c & 1) + g;
      if (slot >= 0)
        a.part[((long long)blockIdx.x * 2 + slot) * kUnit + 32 * warp + in] = mine;
      else if (key0 + in < len)
        a.weights[((long long)ub * a.Hkv + uh) * a.cap + key0 + in] = so_far + mine;
    }
  }
  if (tid == 0) a.begun[blockIdx.x] = begun, a.went_on[blockIdx.x] = went_on;
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

}  // namespace

size_t kv_weights_i4_workspace_bytes() {
  return (size_t)kPerSm * num_sms() * (2 * kUnit * 4 + 32);
}

cudaError_t launch_kv_weights_i4(const uint16_t* q, long long q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                                 long long pages, int ps, const int* table, int width, const int* cu, const int* kv_lens, int B,
                                 float scale, const float* lse, float* weights, void* workspace, unsigned* dev_err,
                                 cudaStream_t s) {
  const int ctas = kPerSm * num_sms();
  float* part = static_cast<float*>(workspace);
  int4* begun = reinterpret_cast<int4*>(part + (size_t)ctas * 2 * kUnit);
  Args a{reinterpret_cast<const __half*>(q), q_stride, T, Hq, Hkv, Hq / Hkv, fast_div(Hq / Hkv), cache, (int)pages,
         ps / kKvBlock, fast_div(ps / kKvBlock), table, width, width * ps, cu, kv_lens, B, scale * kLog2e, lse, weights, begun,
         reinterpret_cast<int*>(begun + ctas), part, dev_err};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = D == 128 ? cudaLaunchKernelEx(&cfg, kv_weights_i4_kernel<128>, a)
                                 : cudaLaunchKernelEx(&cfg, kv_weights_i4_kernel<64>, a);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kUnit, 1, 1);
  return cudaLaunchKernelEx(&cfg, kv_weights_join_kernel, a, ctas);
}

}  // namespace wql
