// kv_weights_i4.cu -- the attention weight that every cached token gets from packed chunks of rows, added to running sums:
//   weights[b, kvh, t] += sum over the rows r of sequence b that see t, and the query heads h of kvh's group, of
//                         exp(scale q[r, h] . k[t] - lse[r, h]),   k = code * s + lo, rounded to fp16.
//
// A CTA takes 64 tokens of a K/V head, a lane two of them; its warps take the rows in turn and their sums are added at the
// end, in a fixed order.
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kKeys = 64, kThreads = 256, kWarps = kThreads / 32;

struct Args {
  const __half* q;
  long long q_stride;
  int T, Hq, Hkv, G;
  const uint8_t* cache;
  int pages, ps;
  FastDiv by_ps;
  const int* table;
  int width, cap;
  const int *cu, *kv_lens;
  float scale;
  const float* lse;
  float* weights;
  unsigned* err;
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv_weights_i4_kernel(const Args a) {
  using L = KvI4<D>;
  constexpr int kPitch = D + 8;
  __shared__ __align__(16) __half ks[kKeys][kPitch];
  __shared__ float qs[kWarps][D], sums[kWarps][kKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.z, kvh = blockIdx.y;
  const KvChunk c = kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, a.err);
  if (c.rows == 0) return;
  for (int t0 = blockIdx.x * kKeys; t0 < c.len; t0 += gridDim.x * kKeys) {
    __syncthreads();
    for (int i = tid; i < kKeys * (D / 8); i += kThreads) {
      const int row = i / (D / 8), ch = i % (D / 8), t = t0 + row;
      uint32_t v[4] = {0u, 0u, 0u, 0u};
      if (t < c.len) {
        const int pg = (int)quot((uint32_t)t, a.by_ps), at = t - pg * a.ps, page = a.table[(long long)b * a.width + pg];
        if (page < 0 || page >= a.pages) {
          report_error(a.err, kErrBadIndex);
        } else {
          const uint8_t* blk = a.cache + (((long long)page * a.Hkv + kvh) * (a.ps / kKvBlock) + at / kKvBlock) * L::kBytes;
          const int rr = at % kKvBlock;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + rr * L::kRow + 4 * ch);
          const uint32_t par = *reinterpret_cast<const uint32_t*>(blk + L::kKp + 4 * rr);
          kv_values8(w, prmt(par, 0, 0x1010), prmt(par, 0, 0x3232), v);
          if (kv_finite(par) && kv_overflows(par))
            for (int j = 0; j < 4; ++j) v[j] = kv_clamp2(v[j]);
        }
      }
      *reinterpret_cast<uint4*>(&ks[row][8 * ch]) =
          make_uint4(prmt(v[0], v[1], 0x5410), prmt(v[2], v[3], 0x5410), prmt(v[0], v[1], 0x7632), prmt(v[2], v[3], 0x7632));
    }
    __syncthreads();
    float sum[2] = {0.f, 0.f};
    const long long rows = (long long)c.rows * a.G;
    for (long long r = (long long)max(t0 - c.first, 0) * a.G + warp; r < rows; r += kWarps) {
      const int tok = (int)(r / a.G), h = kvh * a.G + (int)(r % a.G), last = c.first + tok;
      __syncwarp();
      for (int d = lane; d < D; d += 32) qs[warp][d] = __half2float(a.q[(c.start + tok) * a.q_stride + (long long)h * D + d]);
      __syncwarp();
      float s0 = 0.f, s1 = 0.f;
      for (int d = 0; d < D; ++d) {
        s0 = fmaf(qs[warp][d], __half2float(ks[lane][d]), s0);
        s1 = fmaf(qs[warp][d], __half2float(ks[lane + 32][d]), s1);
      }
      const float z = a.lse[(long long)(c.start + tok) * a.Hq + h];
      if (t0 + lane <= last) sum[0] += expf(s0 * a.scale - z);
      if (t0 + lane + 32 <= last) sum[1] += expf(s1 * a.scale - z);
    }
    sums[warp][lane] = sum[0], sums[warp][lane + 32] = sum[1];
    __syncthreads();
    if (tid < kKeys && t0 + tid < c.len) {
      float x = 0.f;
      for (int w = 0; w < kWarps; ++w) x += sums[w][tid];
      a.weights[((long long)b * a.Hkv + kvh) * a.cap + t0 + tid] += x;
    }
  }
}

}  // namespace

cudaError_t launch_kv_weights_i4(const uint16_t* q, long long q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                                 long long pages, int ps, const int* table, int width, const int* cu, const int* kv_lens, int B,
                                 float scale, const float* lse, float* weights, unsigned* dev_err, cudaStream_t s,
                                 std::string*) {
  Args a{reinterpret_cast<const __half*>(q), q_stride, T, Hq, Hkv, Hq / Hkv, cache, (int)pages, ps, fast_div(ps), table,
         width, width * ps, cu, kv_lens, scale, lse, weights, dev_err};
  const int tiles = (a.cap + kKeys - 1) / kKeys;
  const dim3 grid(tiles < 1024 ? tiles : 1024, Hkv, B);
  if (D == 128)
    kv_weights_i4_kernel<128><<<grid, kThreads, 0, s>>>(a);
  else
    kv_weights_i4_kernel<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace wql
