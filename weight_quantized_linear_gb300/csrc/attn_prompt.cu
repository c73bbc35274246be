// attn_prompt.cu -- causal attention over packed prompts, fp16, grouped heads.
//
// For every sequence i (rows cu[i] .. cu[i + 1] - 1 of q, k and v) and head h, row r:
//   o[r] = sum_{j <= r} softmax_j(scale q[r] . k[j]) v[j],  k and v those of head h / (Hq / Hkv)
// One pass over the keys with the running maximum and sum of the softmax in fp32.
//
// A CTA takes kTileQ query rows of one head; four warps of 16 rows each; key tiles of kTileK rows in shared
// memory, products with mma.sync.
#include <climits>

#include "internal.h"
#include "common.cuh"

namespace wql {
namespace {

constexpr int kTileQ = 64, kTileK = 64, kThreads = 128;

struct Args {
  const __half *q, *k, *v;
  long long qs, ks, vs;  // elements between tokens
  const int* cu;
  int B, T, Hq, Hkv, G;
  float scale_log2;
  __half* out;
  unsigned* err;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_prompt_kernel(const Args a) {
  constexpr int kPitch = D + 8;  // halves per row in shared memory: 16 bytes off a multiple of 128
  __shared__ __align__(16) __half sk[kTileK * kPitch], sv[kTileK * kPitch];
  __shared__ int bad[D];  // first key row whose V value of this channel is not finite
  __shared__ int s_sum[kThreads / 32];
  __shared__ int3 s_tile;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;

  // ---- the sequence and first row of this CTA's tile, counted from the last one ----
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  auto seq = [&](int b, int& start) {
    const int s = a.cu[b], e = a.cu[b + 1];
    if (s < 0 || e < s || e > a.T) {
      report_error(a.err, kErrBadIndex);
      start = 0;
      return 0;
    }
    start = s;
    return e - s;
  };
  int mine = 0, start;
  for (int b = b0; b < b1; ++b) mine += (seq(b, start) + kTileQ - 1) / kTileQ;
  int incl = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (tid == 0) s_tile = make_int3(0, 0, 0);
  __syncthreads();
  int total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) incl += s_sum[w];
    total += s_sum[w];
  }
  const int want = total - 1 - (int)blockIdx.x;
  if (want < 0) return;
  int first = incl - mine;
  if (first <= want && want < incl)
    for (int b = b0; b < b1; ++b) {
      const int len = seq(b, start), n = (len + kTileQ - 1) / kTileQ;
      if (want < first + n) {
        s_tile = make_int3(start, len, (want - first) * kTileQ);
        break;
      }
      first += n;
    }
  for (int i = tid; i < D; i += kThreads) bad[i] = INT_MAX;
  __syncthreads();
  start = s_tile.x;
  const int len = s_tile.y, q0 = s_tile.z, head = blockIdx.y, kvh = head / a.G;

  // Q fragments: rows q0 + 16 warp + g and + 8
  uint32_t qf[D / 16][4];
  const int r0 = q0 + 16 * warp + g;
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 8 * (e & 1);
      qf[j][e] = r < len ? *reinterpret_cast<const uint32_t*>(a.q + (long long)(start + r) * a.qs + (long long)head * D +
                                                            16 * j + 2 * c + 8 * (e >> 1))
                         : 0u;
    }
  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  float m[2] = {-1e30f, -1e30f}, l[2] = {0.f, 0.f};

  const int last = min(q0 + kTileQ, len);
  for (int k0 = 0; k0 < last; k0 += kTileK) {
    __syncthreads();
    for (int i = tid; i < kTileK * D / 8; i += kThreads) {
      const int row = i / (D / 8), ch = i % (D / 8) * 8, j = k0 + row;
      uint4 kk = make_uint4(0u, 0u, 0u, 0u), vv = kk;
      if (j < len) {
        kk = *reinterpret_cast<const uint4*>(a.k + (long long)(start + j) * a.ks + (long long)kvh * D + ch);
        vv = *reinterpret_cast<const uint4*>(a.v + (long long)(start + j) * a.vs + (long long)kvh * D + ch);
      }
      __half* vh = reinterpret_cast<__half*>(&vv);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((__half_as_ushort(vh[e]) & 0x7c00) == 0x7c00) {  // rows before j must not meet 0 * inf
          atomicMin(&bad[ch + e], j);
          vh[e] = __ushort_as_half(0);
        }
      *reinterpret_cast<uint4*>(sk + row * kPitch + ch) = kk;
      *reinterpret_cast<uint4*>(sv + row * kPitch + ch) = vv;
    }
    __syncthreads();
    float s[kTileK / 8][4];
#pragma unroll
    for (int n = 0; n < kTileK / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int n = 0; n < kTileK / 16; ++n) {
        uint32_t x0, x1, x2, x3;  // two 8-key tiles
        ldmatrix_x4(smem_u32(sk + (16 * n + (lane & 7) + ((lane >> 4) << 3)) * kPitch + 16 * j + ((lane >> 3) & 1) * 8), x0,
                    x1, x2, x3);
        mma_f16_16816(s[2 * n], qf[j], x0, x1);
        mma_f16_16816(s[2 * n + 1], qf[j], x2, x3);
      }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < kTileK / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = k0 + 8 * n + 2 * c + (e & 1), row = r0 + 8 * (e >> 1);
        s[n][e] = key <= row ? s[n][e] * a.scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      const float f = ex2(m[e] - mx[e]);
      m[e] = mx[e];
      l[e] *= f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][2 * e] *= f, o[i][2 * e + 1] *= f;
    }
#pragma unroll
    for (int n = 0; n < kTileK / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = ex2(s[n][e] - m[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int n = 0; n < kTileK / 16; ++n) {
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 h = __floats2half2_rn(s[2 * n + (e >> 1)][2 * (e & 1)], s[2 * n + (e >> 1)][2 * (e & 1) + 1]);
        p[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t x0, x1, x2, x3;
        ldmatrix_x4_trans(smem_u32(sv + (16 * n + (lane & 15)) * kPitch + 16 * i + (lane >> 4) * 8), x0, x1, x2, x3);
        mma_f16_16816(o[2 * i], p, x0, x1);
        mma_f16_16816(o[2 * i + 1], p, x2, x3);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int r = r0 + 8 * e;
    if (r >= len) continue;
    const float inv = 1.f / l[e];
    __half* dst = a.out + ((long long)(start + r) * a.Hq + head) * D;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const int ch = 8 * i + 2 * c;
      const float x = r >= bad[ch] ? NAN : o[i][2 * e] * inv, y = r >= bad[ch + 1] ? NAN : o[i][2 * e + 1] * inv;
      *reinterpret_cast<__half2*>(dst + ch) = __floats2half2_rn(x, y);
    }
  }
}

}  // namespace

cudaError_t launch_attn_prompt(const uint16_t* q, long long q_stride, const uint16_t* k, long long k_stride,
                               const uint16_t* v, long long v_stride, int T, int Hq, int Hkv, int D, const int* cu, int B,
                               float scale, uint16_t* out, unsigned* dev_err, cudaStream_t s, std::string* err) {
  (void)err;
  Args a{reinterpret_cast<const __half*>(q), reinterpret_cast<const __half*>(k), reinterpret_cast<const __half*>(v),
         q_stride, k_stride, v_stride, cu, B, T, Hq, Hkv, Hq / Hkv, scale * 1.4426950408889634f,
         reinterpret_cast<__half*>(out), dev_err};
  // no sequence starts more than one ragged tile
  const dim3 grid((unsigned)(T / kTileQ + (B < T ? B : T)), (unsigned)Hq);
  if (D == 128)
    attn_prompt_kernel<128><<<grid, kThreads, 0, s>>>(a);
  else
    attn_prompt_kernel<64><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace wql
