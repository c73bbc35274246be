// api.cu -- the extern "C" entry points declared in include/wql.h: argument validation, kernel
// selection by shape, launch-error reporting and the per-device error word of bounded waits.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "common.cuh"
#include "internal.h"
#include "trace.cuh"
#include "wql.h"

namespace {

thread_local std::string g_last_error;

// One error word per device (this module's copy on each device that loads the library).
__device__ unsigned g_wql_device_error;

unsigned* device_error_word() {
  static std::atomic<unsigned*> cache[64];  // racing first calls store the same address
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  unsigned* w = cache[dev].load(std::memory_order_acquire);
  if (!w) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_wql_device_error) != cudaSuccess) return nullptr;
    w = static_cast<unsigned*>(p);
    cache[dev].store(w, std::memory_order_release);
  }
  return w;
}

// One thread waits on an mbarrier that nothing will complete.  The bounded wait gives up after its
// time limit and records kErrTimeoutFull, exactly as a real kernel does when a copy never lands.
__global__ void expire_wait_kernel(unsigned* err) {
  __shared__ __align__(8) uint64_t bar;
  wql::mbar_init(&bar, 1);  // one arrival expected, none will come
  wql::fence_mbarrier_init();
  if (!wql::mbar_wait_bounded(&bar, 0)) wql::report_error(err, wql::kErrTimeoutFull);
}

wql_status fail(wql_status st, const std::string& msg) {
  g_last_error = msg;
  return st;
}

wql_status cuda_status(cudaError_t e, const char* what, const std::string& extra = std::string()) {
  if (e == cudaSuccess) {
    g_last_error.clear();
    return WQL_OK;
  }
  std::string msg = std::string(what) + ": " + cudaGetErrorString(e);
  if (!extra.empty()) msg += " (" + extra + ")";
  return fail(WQL_ECUDA, msg);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define WQL_REQUIRE(cond, msg)                      \
  do {                                              \
    if (!(cond)) return fail(WQL_EINVAL, (msg));    \
  } while (0)

#define WQL_REQUIRE_PTR(p) WQL_REQUIRE((p) != nullptr && aligned16(p), #p " must be a non-null 16-byte aligned device pointer")

bool valid_group(int g) { return g == 32 || g == 64 || g == 128; }

}  // namespace

void wql::set_last_error(const std::string& msg) { g_last_error = msg; }

extern "C" {

const char* wql_status_string(int status) {
  switch (status) {
    case WQL_OK:
      return "ok";
    case WQL_EINVAL:
      return "invalid argument";
    case WQL_EUNSUPPORTED:
      return "unsupported request";
    case WQL_ECUDA:
      return "CUDA error";
    case WQL_ETIMEOUT:
      return "device-side wait timed out";
    default:
      return "unknown status";
  }
}

const char* wql_last_error(void) { return g_last_error.c_str(); }

int wql_version(void) { return 100; }

wql_status wql_device_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_status(e, "wql_device_status: stream synchronize");
  unsigned* w = device_error_word();
  if (!w) return fail(WQL_ECUDA, "wql_device_status: cannot locate the device error word");
  unsigned v = 0;
  e = cudaMemcpy(&v, w, sizeof(v), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_status(e, "wql_device_status: read error word");
  if (v != 0) {
    const unsigned zero = 0;
    cudaMemcpy(w, &zero, sizeof(zero), cudaMemcpyHostToDevice);
    if (v == wql::kErrBadIndex)
      return fail(WQL_EINVAL, "a kernel met a page, slot or length out of range and left it out");
    char buf[96];
    snprintf(buf, sizeof(buf), "a kernel abandoned a bounded wait (error bits 0x%x)", v);
    return fail(WQL_ETIMEOUT, buf);
  }
  g_last_error.clear();
  return WQL_OK;
}

wql_status wql_awq_pack(const float* w, int K, int N, int group, uint32_t* qweight, uint16_t* scales,
                        uint32_t* qzeros, void* stream) {
  WQL_REQUIRE(valid_group(group), "group must be 32, 64 or 128");
  WQL_REQUIRE(K >= group && K % group == 0, "K must be a positive multiple of the group size");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE_PTR(w);
  WQL_REQUIRE_PTR(qweight);
  WQL_REQUIRE_PTR(scales);
  WQL_REQUIRE_PTR(qzeros);
  return cuda_status(wql::launch_awq_pack(w, K, N, group, qweight, scales, qzeros, static_cast<cudaStream_t>(stream)),
                     "wql_awq_pack");
}

namespace {

// wql_w4a16_gemm and wql_w4a16_gemm_silu_mul: one validation and dispatch path.
wql_status w4a16_gemm(const char* fn, const uint16_t* x, const uint32_t* qweight, const uint16_t* scales,
                      const uint32_t* qzeros, int M, int K, int N, int group, uint16_t* y, int act, void* stream) {
  WQL_REQUIRE(valid_group(group), "group must be 32, 64 or 128");
  WQL_REQUIRE(K >= group && K % group == 0, "K must be a positive multiple of the group size");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE(!act || N % 64 == 0, "N must be a multiple of 64 for the gate/up activation");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(x);
  WQL_REQUIRE_PTR(qweight);
  WQL_REQUIRE_PTR(scales);
  WQL_REQUIRE_PTR(qzeros);
  WQL_REQUIRE_PTR(y);
  unsigned* dev_err = device_error_word();
  std::string err;
  const char* force = getenv("WQL_FORCE_KERNEL");  // benchmarking switch: "decode" or "prefill"
  const bool prefill = force && strcmp(force, "decode") == 0   ? false
                       : force && strcmp(force, "prefill") == 0 ? true
                                                                : wql::w4a16_use_prefill(M, K, N, group);
  cudaError_t e = prefill ? wql::launch_w4a16_prefill(x, qweight, scales, qzeros, M, K, N, group, y, act, dev_err,
                                                      static_cast<cudaStream_t>(stream), &err)
                          : wql::launch_w4a16_decode(x, qweight, scales, qzeros, M, K, N, group, y, act, dev_err,
                                                     static_cast<cudaStream_t>(stream), &err);
  if (!err.empty()) return fail(WQL_ECUDA, std::string(fn) + ": " + err);
  return cuda_status(e, fn);
}

}  // namespace

wql_status wql_w4a16_gemm(const uint16_t* x, const uint32_t* qweight, const uint16_t* scales,
                          const uint32_t* qzeros, int M, int K, int N, int group, uint16_t* y, void* stream) {
  return w4a16_gemm("wql_w4a16_gemm", x, qweight, scales, qzeros, M, K, N, group, y, 0, stream);
}

wql_status wql_w4a16_gemm_silu_mul(const uint16_t* x, const uint32_t* qweight, const uint16_t* scales,
                                   const uint32_t* qzeros, int M, int K, int N, int group, uint16_t* y,
                                   void* stream) {
  return w4a16_gemm("wql_w4a16_gemm_silu_mul", x, qweight, scales, qzeros, M, K, N, group, y, 1, stream);
}

int wql_w4a16_kernel_for(int M, int K, int N, int group) { return wql::w4a16_use_prefill(M, K, N, group) ? 1 : 0; }

wql_status wql_qrmsnorm_quant_i8(const uint16_t* x, const uint16_t* gamma, float eps, int M, int K, int8_t* q,
                                 float* xs, void* stream) {
  WQL_REQUIRE(K >= 8 && K % 8 == 0, "K must be a positive multiple of 8");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (K > 16384) return fail(WQL_EUNSUPPORTED, "K > 16384 is not supported by the register-resident row kernel");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(x);
  WQL_REQUIRE_PTR(gamma);
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  return cuda_status(wql::launch_qrmsnorm_quant_i8(x, gamma, eps, M, K, q, xs, device_error_word(),
                                                   static_cast<cudaStream_t>(stream)),
                     "wql_qrmsnorm_quant_i8");
}

wql_status wql_add_qrmsnorm_quant_i8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, float eps,
                                     int M, int K, uint16_t* residual_out, int8_t* q, float* xs, void* stream) {
  WQL_REQUIRE(K >= 8 && K % 8 == 0, "K must be a positive multiple of 8");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (K > 16384) return fail(WQL_EUNSUPPORTED, "K > 16384 is not supported by the register-resident row kernel");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(x);
  WQL_REQUIRE_PTR(residual);
  WQL_REQUIRE_PTR(gamma);
  WQL_REQUIRE_PTR(residual_out);
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  return cuda_status(wql::launch_add_qrmsnorm_quant_i8(x, residual, gamma, eps, M, K, residual_out, q, xs,
                                                       device_error_word(), static_cast<cudaStream_t>(stream)),
                     "wql_add_qrmsnorm_quant_i8");
}

namespace {

// Shared argument checks of the QRMSNorm entry points (residual and residual_out only when fused).
wql_status norm_args(const uint16_t* x, const uint16_t* gamma, int M, int K, const void* q, const float* xs,
                     bool fused, const uint16_t* residual, const uint16_t* residual_out) {
  WQL_REQUIRE(K >= 8 && K % 8 == 0, "K must be a positive multiple of 8");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (K > 16384) return fail(WQL_EUNSUPPORTED, "K > 16384 is not supported by the register-resident row kernel");
  if (M == 0) return WQL_OK;
  WQL_REQUIRE_PTR(x);
  WQL_REQUIRE_PTR(gamma);
  WQL_REQUIRE_PTR(q);
  if (fused) {
    WQL_REQUIRE_PTR(residual);
    WQL_REQUIRE_PTR(residual_out);
  }
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  return WQL_OK;
}

}  // namespace

namespace {

wql_status per_token_quant(const char* fn, const uint16_t* x, int M, int K, bool fp8, uint8_t* q, float* xs,
                           void* stream) {
  WQL_REQUIRE(K >= 8 && K % 8 == 0, "K must be a positive multiple of 8");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (K > 16384) return fail(WQL_EUNSUPPORTED, "K > 16384 is not supported by the register-resident row kernel");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(x);
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  return cuda_status(wql::launch_per_token_quant(x, M, K, fp8, q, xs, device_error_word(),
                                                 static_cast<cudaStream_t>(stream)),
                     fn);
}

}  // namespace

wql_status wql_per_token_quant_i8(const uint16_t* x, int M, int K, int8_t* q, float* xs, void* stream) {
  return per_token_quant("wql_per_token_quant_i8", x, M, K, false, reinterpret_cast<uint8_t*>(q), xs, stream);
}

wql_status wql_per_token_quant_fp8(const uint16_t* x, int M, int K, uint8_t* q, float* xs, void* stream) {
  return per_token_quant("wql_per_token_quant_fp8", x, M, K, true, q, xs, stream);
}

wql_status wql_qrmsnorm_quant_fp8(const uint16_t* x, const uint16_t* gamma, float eps, int M, int K, uint8_t* q,
                                  float* xs, void* stream) {
  const wql_status st = norm_args(x, gamma, M, K, q, xs, false, nullptr, nullptr);
  if (st != WQL_OK || M == 0) {
    if (st == WQL_OK) g_last_error.clear();
    return st;
  }
  return cuda_status(wql::launch_qrmsnorm_quant_fp8(x, nullptr, gamma, eps, M, K, nullptr, q, xs, device_error_word(),
                                                    static_cast<cudaStream_t>(stream)),
                     "wql_qrmsnorm_quant_fp8");
}

wql_status wql_add_qrmsnorm_quant_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, float eps,
                                      int M, int K, uint16_t* residual_out, uint8_t* q, float* xs, void* stream) {
  const wql_status st = norm_args(x, gamma, M, K, q, xs, true, residual, residual_out);
  if (st != WQL_OK || M == 0) {
    if (st == WQL_OK) g_last_error.clear();
    return st;
  }
  return cuda_status(wql::launch_qrmsnorm_quant_fp8(x, residual, gamma, eps, M, K, residual_out, q, xs,
                                                    device_error_word(), static_cast<cudaStream_t>(stream)),
                     "wql_add_qrmsnorm_quant_fp8");
}

size_t wql_w8a8_workspace_bytes(int M, int K, int N) {
  (void)N;
  if (M < wql::kW8A8PrefillMinM || K <= 0) return 0;  // the streaming decode kernel needs no scratch
  return wql::w8a8_prefill_workspace_bytes(M, K);      // fp16 copy of the activation codes
}

namespace {

// wql_w8a8_gemm and wql_w8a8_gemm_fused: one validation and dispatch path.
wql_status w8a8_gemm(const char* fn, const int8_t* q, const float* xs, const int8_t* qw, const float* ws,
                     const uint16_t* bias, const uint16_t* residual, int M, int K, int N, uint16_t* y,
                     int32_t* acc_out, void* workspace, size_t workspace_bytes, void* stream) {
  WQL_REQUIRE(K >= 16 && K % 16 == 0, "K must be a positive multiple of 16");
  WQL_REQUIRE(K <= 131072, "K must be <= 131072 so that the int32 accumulator cannot overflow");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE_PTR(qw);
  WQL_REQUIRE_PTR(ws);
  WQL_REQUIRE_PTR(y);
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  WQL_REQUIRE(acc_out == nullptr || aligned16(acc_out), "acc_out must be NULL or 16-byte aligned");
  WQL_REQUIRE(bias == nullptr || aligned16(bias), "bias must be NULL or 16-byte aligned");
  WQL_REQUIRE(residual == nullptr || aligned16(residual), "residual must be NULL or 16-byte aligned");
  const size_t need = wql_w8a8_workspace_bytes(M, K, N);
  WQL_REQUIRE(workspace_bytes >= need, "workspace is smaller than wql_w8a8_workspace_bytes()");
  WQL_REQUIRE(need == 0 || (workspace != nullptr && aligned16(workspace)), "workspace must be 16-byte aligned");
  unsigned* dev_err = device_error_word();
  std::string err;
  const char* force = getenv("WQL_FORCE_KERNEL");  // benchmarking switch: "decode" or "prefill"
  const bool prefill = force && strcmp(force, "decode") == 0 ? false : M >= wql::kW8A8PrefillMinM;
  cudaError_t e = prefill ? wql::launch_w8a8_prefill(q, xs, qw, ws, M, K, N, y, acc_out, bias, residual, workspace,
                                                     dev_err, static_cast<cudaStream_t>(stream), &err)
                          : wql::launch_w8a8_decode(q, xs, qw, ws, M, K, N, y, acc_out, bias, residual, dev_err,
                                                    static_cast<cudaStream_t>(stream), &err);
  if (!err.empty()) return fail(WQL_ECUDA, std::string(fn) + ": " + err);
  return cuda_status(e, fn);
}

}  // namespace

wql_status wql_w8a8_gemm(const int8_t* q, const float* xs, const int8_t* qw, const float* ws, int M, int K, int N,
                         uint16_t* y, int32_t* acc_out, void* workspace, size_t workspace_bytes, void* stream) {
  return w8a8_gemm("wql_w8a8_gemm", q, xs, qw, ws, nullptr, nullptr, M, K, N, y, acc_out, workspace,
                   workspace_bytes, stream);
}

wql_status wql_w8a8_gemm_fused(const int8_t* q, const float* xs, const int8_t* qw, const float* ws,
                               const uint16_t* bias, const uint16_t* residual, int M, int K, int N, uint16_t* y,
                               int32_t* acc_out, void* workspace, size_t workspace_bytes, void* stream) {
  return w8a8_gemm("wql_w8a8_gemm_fused", q, xs, qw, ws, bias, residual, M, K, N, y, acc_out, workspace,
                   workspace_bytes, stream);
}

wql_status wql_w8a8_gemm_fp8(const uint8_t* q, const float* xs, const uint8_t* qw, const float* ws,
                             const uint16_t* bias, const uint16_t* residual, int M, int K, int N, uint16_t* y,
                             float* acc_out, void* stream) {
  WQL_REQUIRE(K >= 16 && K % 16 == 0, "K must be a positive multiple of 16");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (M == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE_PTR(qw);
  WQL_REQUIRE_PTR(ws);
  WQL_REQUIRE_PTR(y);
  WQL_REQUIRE(xs != nullptr && (reinterpret_cast<uintptr_t>(xs) & 3u) == 0, "xs must be a 4-byte aligned device pointer");
  WQL_REQUIRE(acc_out == nullptr || aligned16(acc_out), "acc_out must be NULL or 16-byte aligned");
  WQL_REQUIRE(bias == nullptr || aligned16(bias), "bias must be NULL or 16-byte aligned");
  WQL_REQUIRE(residual == nullptr || aligned16(residual), "residual must be NULL or 16-byte aligned");
  unsigned* dev_err = device_error_word();
  std::string err;
  const char* force = getenv("WQL_FORCE_KERNEL");  // benchmarking switch: "decode"
  const bool prefill = force && strcmp(force, "decode") == 0 ? false : M >= wql::kFp8PrefillMinM;
  cudaError_t e = prefill ? wql::launch_fp8_prefill(q, xs, qw, ws, M, K, N, y, acc_out, bias, residual, dev_err,
                                                    static_cast<cudaStream_t>(stream), &err)
                          : wql::launch_fp8_decode(q, xs, qw, ws, M, K, N, y, acc_out, bias, residual, dev_err,
                                                   static_cast<cudaStream_t>(stream), &err);
  if (!err.empty()) return fail(WQL_ECUDA, "wql_w8a8_gemm_fp8: " + err);
  return cuda_status(e, "wql_w8a8_gemm_fp8");
}

wql_status wql_act_absmax(const uint16_t* x, const uint16_t* gamma, float eps, int M, int K, float* absmax,
                          void* stream) {
  WQL_REQUIRE(K >= 8 && K % 8 == 0, "K must be a positive multiple of 8");
  WQL_REQUIRE(M >= 0, "M must be >= 0");
  if (K > 16384) return fail(WQL_EUNSUPPORTED, "K > 16384 is not supported by the register-resident row kernel");
  WQL_REQUIRE_PTR(absmax);
  if (M > 0) {
    WQL_REQUIRE_PTR(x);
    WQL_REQUIRE_PTR(gamma);
  }
  return cuda_status(wql::launch_act_absmax(x, gamma, eps, M, K, absmax, device_error_word(),
                                            static_cast<cudaStream_t>(stream)),
                     "wql_act_absmax");
}

wql_status wql_smooth(const float* absmax, const uint16_t* gamma, const float* w, int K, int N, float* s,
                      uint16_t* gamma_out, float* w_out, void* stream) {
  WQL_REQUIRE(K >= 16 && K % 16 == 0, "K must be a positive multiple of 16");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE_PTR(absmax);
  WQL_REQUIRE_PTR(gamma);
  WQL_REQUIRE_PTR(w);
  WQL_REQUIRE_PTR(s);
  WQL_REQUIRE_PTR(gamma_out);
  WQL_REQUIRE_PTR(w_out);
  return cuda_status(wql::launch_smooth(absmax, gamma, w, K, N, s, gamma_out, w_out, static_cast<cudaStream_t>(stream)),
                     "wql_smooth");
}

wql_status wql_per_channel_quant_i8(const float* w, int K, int N, int8_t* qw, float* ws, void* stream) {
  WQL_REQUIRE(K >= 16 && K % 16 == 0, "K must be a positive multiple of 16");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE_PTR(w);
  WQL_REQUIRE_PTR(qw);
  WQL_REQUIRE_PTR(ws);
  return cuda_status(wql::launch_per_channel_quant_i8(w, K, N, qw, ws, static_cast<cudaStream_t>(stream)),
                     "wql_per_channel_quant_i8");
}

wql_status wql_per_channel_quant_fp8(const float* w, int K, int N, uint8_t* qw, float* ws, void* stream) {
  WQL_REQUIRE(K >= 16 && K % 16 == 0, "K must be a positive multiple of 16");
  WQL_REQUIRE(N >= 32 && N % 32 == 0, "N must be a positive multiple of 32");
  WQL_REQUIRE_PTR(w);
  WQL_REQUIRE_PTR(qw);
  WQL_REQUIRE_PTR(ws);
  return cuda_status(wql::launch_per_channel_quant_fp8(w, K, N, qw, ws, static_cast<cudaStream_t>(stream)),
                     "wql_per_channel_quant_fp8");
}

wql_status wql_kv_quant_i8(const uint16_t* kv, int64_t rows, int D, int8_t* q, float* scales, void* stream) {
  WQL_REQUIRE(D >= 128 && D % 128 == 0, "D must be a positive multiple of 128");
  WQL_REQUIRE(rows >= 0, "rows must be >= 0");
  if (rows == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(kv);
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(scales != nullptr && (reinterpret_cast<uintptr_t>(scales) & 3u) == 0,
              "scales must be a 4-byte aligned device pointer");
  return cuda_status(wql::launch_kv_quant_i8(kv, rows, D, q, scales, static_cast<cudaStream_t>(stream)),
                     "wql_kv_quant_i8");
}

wql_status wql_kv_dequant_i8(const int8_t* q, const float* scales, int64_t rows, int D, uint16_t* out, void* stream) {
  WQL_REQUIRE(D >= 128 && D % 128 == 0, "D must be a positive multiple of 128");
  WQL_REQUIRE(rows >= 0, "rows must be >= 0");
  if (rows == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE_PTR(out);
  WQL_REQUIRE(scales != nullptr && (reinterpret_cast<uintptr_t>(scales) & 3u) == 0,
              "scales must be a 4-byte aligned device pointer");
  return cuda_status(wql::launch_kv_dequant_i8(q, scales, rows, D, out, static_cast<cudaStream_t>(stream)),
                     "wql_kv_dequant_i8");
}

namespace {

bool kv_head_dim(int D) { return D == 64 || D == 128; }

// Scores of fp16 rows stay below 2^(64 + 39), far inside fp32's range, and the kernels' factors beside the scale too.
bool valid_scale(float scale) { return std::fabs(scale) <= 18446744073709551616.f; }

// Rows [T, H, D] with `stride` elements between tokens, loaded 16 bytes at a time.
bool valid_stride(int64_t stride, int H, int D) { return stride >= (int64_t)H * D && stride % 8 == 0; }

#define WQL_REQUIRE_PTR4(p) \
  WQL_REQUIRE((p) != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0, #p " must be a non-null 4-byte aligned device pointer")

#define WQL_REQUIRE_CACHE()                                                                                        \
  do {                                                                                                             \
    if (!kv_head_dim(D)) return fail(WQL_EUNSUPPORTED, "D must be 64 or 128");                                     \
    WQL_REQUIRE(page_size >= 16 && page_size % 16 == 0, "page_size must be a positive multiple of 16");            \
    WQL_REQUIRE(pages >= 1 && pages * page_size <= INT_MAX, "pages * page_size must be between 16 and 2^31 - 1");  \
  } while (0)

}  // namespace

wql_status wql_kv_plan_pages(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                             const int32_t* free_pages, int free_capacity, const int32_t* free_count,
                             int32_t* block_table, int table_width, int T, int32_t* cu_new, int32_t* kv_lens,
                             int32_t* slots, int32_t* free_count_out, void* stream) {
  WQL_REQUIRE(B >= 0 && T >= 0, "B and T must be >= 0");
  if (B > wql::kPlanMaxB) return fail(WQL_EUNSUPPORTED, "B must be at most 4096");
  WQL_REQUIRE(page_size >= 16 && page_size % 16 == 0, "page_size must be a positive multiple of 16");
  WQL_REQUIRE(table_width >= 1 && (int64_t)table_width * page_size <= INT_MAX,
              "table_width * page_size must be between 16 and 2^31 - 1");
  WQL_REQUIRE(free_capacity >= 0, "free_capacity must be >= 0");
  WQL_REQUIRE_PTR4(free_count);
  WQL_REQUIRE_PTR4(free_count_out);
  WQL_REQUIRE(free_count != free_count_out, "free_count_out must not be free_count");
  WQL_REQUIRE_PTR4(cu_new);
  WQL_REQUIRE(T == 0 || (slots != nullptr && aligned16(slots)), "slots must be a non-null 16-byte aligned device pointer");
  WQL_REQUIRE(free_capacity == 0 || free_pages != nullptr, "free_pages must not be null");
  if (B > 0) {
    WQL_REQUIRE_PTR4(ctx_lens);
    WQL_REQUIRE_PTR4(new_lens);
    WQL_REQUIRE_PTR4(block_table);
    WQL_REQUIRE_PTR4(kv_lens);
  }
  return cuda_status(wql::launch_kv_plan(ctx_lens, new_lens, B, page_size, free_pages, free_capacity, free_count,
                                         block_table, table_width, T, cu_new, kv_lens, slots, free_count_out,
                                         static_cast<cudaStream_t>(stream)),
                     "wql_kv_plan_pages");
}

wql_status wql_kv_append_i4(const uint16_t* k, const uint16_t* v, int64_t k_stride, int64_t v_stride, int T, int H,
                            int D, const int32_t* slots, uint8_t* cache, int64_t pages, int page_size, void* stream) {
  WQL_REQUIRE(T >= 0, "T must be >= 0");
  WQL_REQUIRE(H >= 1, "H must be >= 1");
  WQL_REQUIRE_CACHE();
  if ((int64_t)T * H > INT_MAX) return fail(WQL_EUNSUPPORTED, "T * H must be below 2^31");
  if (T == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(k);
  WQL_REQUIRE_PTR(v);
  WQL_REQUIRE(valid_stride(k_stride, H, D) && valid_stride(v_stride, H, D),
              "token strides must be multiples of 8 and at least H * D");
  WQL_REQUIRE_PTR4(slots);
  WQL_REQUIRE_PTR(cache);
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_kv_append_i4: cannot locate the device error word");
  return cuda_status(wql::launch_kv_append_i4(k, v, k_stride, v_stride, T, H, D, slots, cache, pages, page_size, dev_err,
                                              static_cast<cudaStream_t>(stream)),
                     "wql_kv_append_i4");
}

wql_status wql_kv_read_i4(const uint8_t* cache, int64_t pages, int page_size, int H, int D, const int32_t* slots, int T,
                          uint16_t* k, uint16_t* v, void* stream) {
  WQL_REQUIRE(T >= 0, "T must be >= 0");
  WQL_REQUIRE(H >= 1, "H must be >= 1");
  WQL_REQUIRE_CACHE();
  if ((int64_t)T * H > INT_MAX) return fail(WQL_EUNSUPPORTED, "T * H must be below 2^31");
  if (T == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(cache);
  WQL_REQUIRE_PTR4(slots);
  WQL_REQUIRE_PTR(k);
  WQL_REQUIRE_PTR(v);
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_kv_read_i4: cannot locate the device error word");
  return cuda_status(wql::launch_kv_read_i4(cache, pages, page_size, H, D, slots, T, k, v, dev_err,
                                            static_cast<cudaStream_t>(stream)),
                     "wql_kv_read_i4");
}

size_t wql_attention_kv_i4_workspace_bytes(int B, int Lq, int Hq, int Hkv, int D) {
  if (B < 1 || Lq < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || !kv_head_dim(D)) return 0;
  return wql::attn_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D);
}

wql_status wql_attention_kv_i4(const uint16_t* q, int64_t q_stride, int B, int Lq, int Hq, int Hkv, int D,
                               const uint8_t* cache, int64_t pages, int page_size, const int32_t* block_table,
                               int table_width, const int32_t* kv_lens, float scale, uint16_t* out, void* workspace,
                               size_t workspace_bytes, void* stream) {
  WQL_REQUIRE(B >= 0 && Lq >= 0, "B and Lq must be >= 0");
  WQL_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0, "Hq must be a positive multiple of Hkv");
  WQL_REQUIRE_CACHE();
  WQL_REQUIRE(table_width >= 1 && (int64_t)table_width * page_size <= INT_MAX,
              "table_width * page_size must be between 16 and 2^31 - 1");
  WQL_REQUIRE((int64_t)Lq * Hq <= INT_MAX / 256, "Lq * Hq is too large");
  WQL_REQUIRE(valid_scale(scale), "scale must be finite and at most 2^64 in magnitude");
  // the kernel counts 32-token steps (and a few per K/V head beside them) in 32 bits
  const int64_t row_blocks = ((int64_t)Lq * (Hq / Hkv) + 7) / 8, steps = ((int64_t)table_width * page_size + 31) / 32 + 4;
  if ((double)B * Hkv * (double)row_blocks * (double)steps > (double)INT_MAX)
    return fail(WQL_EUNSUPPORTED, "B * Hkv * row blocks * (table_width * page_size / 32 + 4) must be below 2^31");
  if (B == 0 || Lq == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(valid_stride(q_stride, Hq, D), "the token stride of q must be a multiple of 8 and at least Hq * D");
  WQL_REQUIRE_PTR(cache);
  WQL_REQUIRE_PTR4(block_table);
  WQL_REQUIRE_PTR4(kv_lens);
  WQL_REQUIRE_PTR(out);
  WQL_REQUIRE_PTR(workspace);
  WQL_REQUIRE(workspace_bytes >= wql::attn_kv_i4_workspace_bytes(B, Lq, Hq, Hkv, D),
              "workspace is smaller than wql_attention_kv_i4_workspace_bytes");
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_attention_kv_i4: cannot locate the device error word");
  std::string err;
  const cudaError_t e = wql::launch_attn_kv_i4(q, q_stride, B, Lq, Hq, Hkv, D, cache, pages, page_size, block_table,
                                               table_width, kv_lens, scale, out, workspace, dev_err,
                                               static_cast<cudaStream_t>(stream), &err);
  return cuda_status(e, "wql_attention_kv_i4", err);
}

wql_status wql_attention_prompt(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                const uint16_t* v, int64_t v_stride, int T, int Hq, int Hkv, int D,
                                const int32_t* cu_seqlens, int B, float scale, uint16_t* out, void* stream) {
  WQL_REQUIRE(T >= 0 && B >= 0, "T and B must be >= 0");
  WQL_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0, "Hq must be a positive multiple of Hkv");
  if (!kv_head_dim(D)) return fail(WQL_EUNSUPPORTED, "D must be 64 or 128");
  if (Hq > 65535) return fail(WQL_EUNSUPPORTED, "Hq must be at most 65535");
  WQL_REQUIRE(valid_scale(scale), "scale must be finite and at most 2^64 in magnitude");
  if (T == 0 || B == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE_PTR(k);
  WQL_REQUIRE_PTR(v);
  WQL_REQUIRE(valid_stride(q_stride, Hq, D) && valid_stride(k_stride, Hkv, D) && valid_stride(v_stride, Hkv, D),
              "token strides must be multiples of 8 and at least heads * D");
  WQL_REQUIRE_PTR4(cu_seqlens);
  WQL_REQUIRE_PTR(out);
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_attention_prompt: cannot locate the device error word");
  std::string err;
  cudaError_t e = wql::launch_attn_prompt(q, q_stride, k, k_stride, v, v_stride, T, Hq, Hkv, D, cu_seqlens, B, scale, out,
                                          dev_err, static_cast<cudaStream_t>(stream), &err);
  return cuda_status(e, "wql_attention_prompt", err);
}

namespace {

// What attention_chunks_kv_i4 and kv_weights_i4 ask of the arguments that they share; *empty: there is nothing to do.
wql_status check_chunks(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                        int64_t pages, int page_size, const int32_t* block_table, int table_width, const int32_t* cu_new,
                        const int32_t* kv_lens, int B, float scale, bool* empty) {
  *empty = false;
  WQL_REQUIRE(T >= 0 && B >= 0, "T and B must be >= 0");
  WQL_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0, "Hq must be a positive multiple of Hkv");
  WQL_REQUIRE_CACHE();
  if (B > wql::kPlanMaxB) return fail(WQL_EUNSUPPORTED, "B must be at most 4096");
  if (Hq > 65535 || Hq / Hkv > 128) return fail(WQL_EUNSUPPORTED, "Hq must be at most 65535 and Hq / Hkv at most 128");
  if ((int64_t)T * Hq > INT_MAX) return fail(WQL_EUNSUPPORTED, "T * Hq must be below 2^31");
  WQL_REQUIRE(table_width >= 1 && (int64_t)table_width * page_size <= INT_MAX,
              "table_width * page_size must be between 16 and 2^31 - 1");
  WQL_REQUIRE(valid_scale(scale), "scale must be finite and at most 2^64 in magnitude");
  if (T == 0 || B == 0) {
    *empty = true;
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(q);
  WQL_REQUIRE(valid_stride(q_stride, Hq, D), "the token stride of q must be a multiple of 8 and at least Hq * D");
  WQL_REQUIRE_PTR(cache);
  WQL_REQUIRE_PTR4(block_table);
  WQL_REQUIRE_PTR4(cu_new);
  WQL_REQUIRE_PTR4(kv_lens);
  return WQL_OK;
}

}  // namespace

size_t wql_attention_chunks_kv_i4_workspace_bytes(int T, int B, int Hq, int Hkv, int D) {
  if (T < 1 || B < 1 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq / Hkv > 128 || !kv_head_dim(D)) return 0;
  return wql::attn_chunks_i4_workspace_bytes(T, B, Hq, Hkv, D);
}

wql_status wql_attention_chunks_kv_i4(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D,
                                      const uint8_t* cache, int64_t pages, int page_size, const int32_t* block_table,
                                      int table_width, const int32_t* cu_new, const int32_t* kv_lens, int B, float scale,
                                      uint16_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty;
  const wql_status st = check_chunks(q, q_stride, T, Hq, Hkv, D, cache, pages, page_size, block_table, table_width, cu_new,
                                     kv_lens, B, scale, &empty);
  if (st != WQL_OK || empty) return st;
  WQL_REQUIRE_PTR(out);
  WQL_REQUIRE((reinterpret_cast<uintptr_t>(lse) & 3u) == 0, "lse must be null or 4-byte aligned");
  WQL_REQUIRE_PTR(workspace);
  WQL_REQUIRE(workspace_bytes >= wql::attn_chunks_i4_workspace_bytes(T, B, Hq, Hkv, D),
              "workspace is smaller than wql_attention_chunks_kv_i4_workspace_bytes");
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_attention_chunks_kv_i4: cannot locate the device error word");
  std::string err;
  const cudaError_t e = wql::launch_attn_chunks_i4(q, q_stride, T, Hq, Hkv, D, cache, pages, page_size, block_table,
                                                   table_width, cu_new, kv_lens, B, scale, out, lse, workspace, dev_err,
                                                   static_cast<cudaStream_t>(stream), &err);
  return cuda_status(e, "wql_attention_chunks_kv_i4", err);
}

size_t wql_kv_weights_i4_workspace_bytes(void) { return wql::kv_weights_i4_workspace_bytes(); }

wql_status wql_kv_weights_i4(const uint16_t* q, int64_t q_stride, int T, int Hq, int Hkv, int D, const uint8_t* cache,
                             int64_t pages, int page_size, const int32_t* block_table, int table_width,
                             const int32_t* cu_new, const int32_t* kv_lens, int B, float scale, const float* lse,
                             float* weights, void* workspace, size_t workspace_bytes, void* stream) {
  bool empty;
  const wql_status st = check_chunks(q, q_stride, T, Hq, Hkv, D, cache, pages, page_size, block_table, table_width, cu_new,
                                     kv_lens, B, scale, &empty);
  if (st != WQL_OK || empty) return st;
  WQL_REQUIRE_PTR4(lse);
  WQL_REQUIRE_PTR(weights);
  WQL_REQUIRE_PTR(workspace);
  WQL_REQUIRE(workspace_bytes >= wql::kv_weights_i4_workspace_bytes(),
              "workspace is smaller than wql_kv_weights_i4_workspace_bytes");
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_kv_weights_i4: cannot locate the device error word");
  std::string err;
  const cudaError_t e = wql::launch_kv_weights_i4(q, q_stride, T, Hq, Hkv, D, cache, pages, page_size, block_table,
                                                  table_width, cu_new, kv_lens, B, scale, lse, weights, workspace, dev_err,
                                                  static_cast<cudaStream_t>(stream), &err);
  return cuda_status(e, "wql_kv_weights_i4", err);
}

wql_status wql_kv_evict_i4(const float* weights, uint8_t* cache, int64_t pages, int page_size, int H, int D,
                           const int32_t* block_table, int table_width, const int32_t* kv_lens, int B,
                           const int32_t* new_table, int new_width, int budget, int recent, int32_t* kept,
                           float* new_weights, int32_t* new_lens, void* stream) {
  WQL_REQUIRE(B >= 0, "B must be >= 0");
  WQL_REQUIRE(H >= 1, "H must be >= 1");
  WQL_REQUIRE_CACHE();
  if (B > wql::kPlanMaxB) return fail(WQL_EUNSUPPORTED, "B must be at most 4096");
  WQL_REQUIRE(table_width >= 1 && (int64_t)table_width * page_size <= INT_MAX,
              "table_width * page_size must be between 16 and 2^31 - 1");
  WQL_REQUIRE(new_width >= 1 && (int64_t)new_width * page_size <= INT_MAX,
              "new_width * page_size must be between 16 and 2^31 - 1");
  WQL_REQUIRE(budget >= 1 && budget <= (int64_t)new_width * page_size, "budget must be between 1 and new_width * page_size");
  WQL_REQUIRE(recent >= 0, "recent must be >= 0");
  if ((int64_t)B * H > INT_MAX / (((int64_t)budget + 15) / 16) || (int64_t)B * H > INT_MAX / 8)
    return fail(WQL_EUNSUPPORTED, "B * H * max(8, ceil(budget / 16)) must be below 2^31");
  if (B == 0) {
    g_last_error.clear();
    return WQL_OK;
  }
  WQL_REQUIRE_PTR(weights);
  WQL_REQUIRE_PTR(cache);
  WQL_REQUIRE_PTR4(block_table);
  WQL_REQUIRE_PTR4(kv_lens);
  WQL_REQUIRE_PTR4(new_table);
  WQL_REQUIRE_PTR4(kept);
  WQL_REQUIRE_PTR(new_weights);
  WQL_REQUIRE_PTR4(new_lens);
  WQL_REQUIRE(new_table != block_table && new_weights != weights && new_lens != kv_lens,
              "new_table, new_weights and new_lens must not be block_table, weights and kv_lens");
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_kv_evict_i4: cannot locate the device error word");
  return cuda_status(wql::launch_kv_evict_i4(weights, cache, pages, page_size, H, D, block_table, table_width, kv_lens, B,
                                             new_table, new_width, budget, recent, kept, new_weights, new_lens, dev_err,
                                             static_cast<cudaStream_t>(stream)),
                     "wql_kv_evict_i4");
}

wql_status wql_diag_expire_wait(void* stream) {
  unsigned* dev_err = device_error_word();
  if (!dev_err) return fail(WQL_ECUDA, "wql_diag_expire_wait: cannot locate the device error word");
  expire_wait_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(dev_err);
  return cuda_status(cudaGetLastError(), "wql_diag_expire_wait");
}

wql_status wql_trace_setup(uint64_t* buf, const void* ybase, uint64_t ystride, int launches, int ctas) {
#ifdef WQL_PHASE_TRACE
  WQL_REQUIRE(buf == nullptr || (launches > 0 && ctas > 0 && ystride > 0 &&
                                 (reinterpret_cast<uintptr_t>(buf) & 7u) == 0),
              "buf must be null, or 8-byte aligned with positive launches, ctas and ystride");
  wql::TraceDesc d{reinterpret_cast<unsigned long long*>(buf), reinterpret_cast<unsigned long long>(ybase),
                   (unsigned long long)ystride, launches, ctas};
  cudaError_t e = wql::trace_set_w4a16_decode(d);
  if (e == cudaSuccess) e = wql::trace_set_w4a16_prefill(d);
  return cuda_status(e, "wql_trace_setup");
#else
  (void)buf;
  (void)ybase;
  (void)ystride;
  (void)launches;
  (void)ctas;
  return fail(WQL_EUNSUPPORTED, "wql_trace_setup: this library was built without WQL_PHASE_TRACE");
#endif
}

}  // extern "C"
