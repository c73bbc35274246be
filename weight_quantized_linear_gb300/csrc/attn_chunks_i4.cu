// attn_chunks_i4.cu -- attention of packed chunks of new tokens over the paged 4-bit KV cache, with grouped heads.
//
// Sequence b's chunk is rows cu[b] .. cu[b + 1] - 1 of q, the last ones of its kv_lens[b] tokens, all of which are in the
// cache.  For row r of n and query head h:
//   out = sum_t softmax_t(scale q . k[t]) v[t],   lse = ln sum_t exp(scale q . k[t]),   t <= kv_len - n + r
// with k and v of K/V head h / (Hq / Hkv): code * s + lo, rounded to fp16.
//
// A CTA takes kRows (token, query head) rows of a K/V head and walks through the keys in tiles of kKeys, dequantised to
// shared memory; a warp owns two rows, a lane two keys of a tile and then D / 32 channels of the output.
#include "internal.h"
#include "kv_i4.cuh"

namespace wql {
namespace {

constexpr int kRows = 16, kKeys = 64, kThreads = 256;

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
  __half* out;
  float* lse;
  unsigned* err;
};

template <int D>
__global__ void __launch_bounds__(kThreads) attn_chunks_i4_kernel(const Args a) {
  using L = KvI4<D>;
  constexpr int kPitch = D + 8;  // halves
  __shared__ __align__(16) __half kv[2][kKeys][kPitch];
  __shared__ float qs[kRows][D], ps[kRows][kKeys];
  __shared__ bool bad[kKeys];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int b = blockIdx.z, kvh = blockIdx.y;
  const KvChunk c = kv_chunk(a.cu, a.kv_lens, b, a.T, a.cap, a.err);
  const long long rows = (long long)c.rows * a.G;
  for (long long r0 = (long long)blockIdx.x * kRows; r0 < rows; r0 += (long long)gridDim.x * kRows) {
    __syncthreads();
    for (int i = tid; i < kRows * D; i += kThreads) {
      const long long r = r0 + i / D;
      float v = 0.f;
      if (r < rows) {
        const int tok = (int)(r / a.G), h = kvh * a.G + (int)(r % a.G);
        v = __half2float(a.q[(c.start + tok) * a.q_stride + (long long)h * D + i % D]);
      }
      qs[i / D][i % D] = v;
    }
    const long long last_row = min(r0 + kRows, rows) - 1;
    const int keys = min(c.len, c.first + (int)(last_row / a.G) + 1);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[2][D / 32] = {};
    for (int t0 = 0; t0 < keys; t0 += kKeys) {
      __syncthreads();
      for (int i = tid; i < 2 * kKeys * (D / 8); i += kThreads) {
        const int is_v = i / (kKeys * (D / 8)), row = i / (D / 8) % kKeys, ch = i % (D / 8), t = t0 + row;
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        bool nan = false;
        if (t < keys) {
          const int pg = (int)quot((uint32_t)t, a.by_ps), at = t - pg * a.ps, page = a.table[(long long)b * a.width + pg];
          if (page < 0 || page >= a.pages) {
            report_error(a.err, kErrBadIndex);
          } else {
            const uint8_t* blk = a.cache + (((long long)page * a.Hkv + kvh) * (a.ps / kKvBlock) + at / kKvBlock) * L::kBytes;
            const int rr = at % kKvBlock;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + (is_v ? L::kV : 0) + rr * L::kRow + 4 * ch);
            const uint32_t par = *reinterpret_cast<const uint32_t*>(blk + (is_v ? L::kVp : L::kKp) + 4 * rr);
            nan = !kv_finite(par);
            kv_values8(w, prmt(par, 0, 0x1010), prmt(par, 0, 0x3232), v);
            if (!nan && kv_overflows(par))
              for (int j = 0; j < 4; ++j) v[j] = kv_clamp2(v[j]);
            if (nan)
              for (int j = 0; j < 4; ++j) v[j] = is_v ? 0u : 0x7fff7fffu;
          }
        }
        if (is_v && ch == 0) bad[row] = nan;
        *reinterpret_cast<uint4*>(&kv[is_v][row][8 * ch]) =
            make_uint4(prmt(v[0], v[1], 0x5410), prmt(v[2], v[3], 0x5410), prmt(v[0], v[1], 0x7632), prmt(v[2], v[3], 0x7632));
      }
      __syncthreads();
      for (int k = 0; k < 2; ++k) {
        const int row = 2 * warp + k;
        const long long r = r0 + row;
        const int last = c.first + (int)(min(r, rows - 1) / a.G);
        float s[2] = {0.f, 0.f};
        for (int d = 0; d < D; ++d) {
          s[0] = fmaf(qs[row][d], __half2float(kv[0][lane][d]), s[0]);
          s[1] = fmaf(qs[row][d], __half2float(kv[0][lane + 32][d]), s[1]);
        }
        bool nan = false;
        for (int j = 0; j < 2; ++j) {
          const int t = t0 + lane + 32 * j;
          s[j] = t <= last ? s[j] * a.scale : -INFINITY;
          nan |= t <= last && bad[lane + 32 * j];
        }
        float top = fmaxf(m[k], fmaxf(s[0], s[1]));
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == -INFINITY ? 0.f : top;
        const float f = __expf(m[k] - base), p0 = __expf(s[0] - base), p1 = __expf(s[1] - base);
        m[k] = top;
        float sum = p0 + p1;
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l[k] = l[k] * f + sum;
        ps[row][lane] = p0, ps[row][lane + 32] = p1;
        const bool any = __any_sync(0xffffffffu, nan);
        __syncwarp();
        for (int i = 0; i < D / 32; ++i) {
          float x = o[k][i] * f;
          for (int t = 0; t < kKeys; ++t) x = fmaf(ps[row][t], __half2float(kv[1][t][lane + 32 * i]), x);
          o[k][i] = any ? NAN : x;
        }
      }
    }
    for (int k = 0; k < 2; ++k) {
      const long long r = r0 + 2 * warp + k;
      if (r >= rows) continue;
      const int tok = (int)(r / a.G), h = kvh * a.G + (int)(r % a.G);
      const bool none = c.first + tok < 0;  // sees nothing
      const long long at = (long long)(c.start + tok) * a.Hq + h;
      for (int i = 0; i < D / 32; ++i) a.out[at * D + lane + 32 * i] = __float2half_rn(none ? 0.f : o[k][i] / l[k]);
      if (a.lse && lane == 0) a.lse[at] = none ? -INFINITY : m[k] + logf(l[k]);
    }
  }
}

}  // namespace

size_t attn_chunks_i4_workspace_bytes(int, int, int, int, int) { return 16; }

cudaError_t launch_attn_chunks_i4(const uint16_t* q, long long q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                                  long long pages, int ps, const int* table, int width, const int* cu, const int* kv_lens,
                                  int B, float scale, uint16_t* out, float* lse, void*, unsigned* dev_err, cudaStream_t s,
                                  std::string*) {
  Args a{reinterpret_cast<const __half*>(q), q_stride, T, Hq, Hkv, Hq / Hkv, cache, (int)pages, ps, fast_div(ps), table,
         width, width * ps, cu, kv_lens, scale, reinterpret_cast<__half*>(out), lse, dev_err};
  const long long tiles = ((long long)T * a.G + kRows - 1) / kRows;
  const dim3 grid((unsigned)(tiles < 256 ? tiles : 256), Hkv, B);
  if (D == 128)
    attn_chunks_i4_kernel<128><<<grid, kThreads, 0, s>>>(a);
  else
    attn_chunks_i4_kernel<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace wql
