// wp_multi.cu -- one shared projection for rows that belong to the requests of many adapters.
//
//   Y[t, g] = X[t] W_g^T + bias_g + s_t (X[t] A_{a,g}^T) B_{a,g}^T,   a = slot[t]
//
// (sglang PR, Motivation: the adapter and its scale belong to the request, so a batch meets
// many of them.)  The adapters of a layer lie in a bank, one per slot, and every row names its
// slot on the device.
//
// First form: the plain projection in fp32, then H~ = bf16(s X A^T) a warp per rank row, then
// the second contraction added before the single output rounding.
#include <cmath>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }

__global__ void __launch_bounds__(256) multi_h_kernel(const MultiCall p) {
  const int t = blockIdx.x;
  const int a = p.slot[t];
  const int lane = threadIdx.x & 31;
  float s = 0.f;
  if (a >= 0 && a < p.S) {
    s = p.scale[a];
    if (p.row_scale) s = __fmul_rn(s, p.row_scale[t]);
    s = __fmul_rn(s, p.request_scale);
  }
  const uint16_t* x = p.X + static_cast<long long>(t) * p.ldx;
  for (int j = threadIdx.x >> 5; j < p.G * p.R16; j += 8) {
    const int g = j / p.R16, r = j - g * p.R16;
    float h = 0.f;
    if (s != 0.f && r < p.R) {
      const uint16_t* ar = p.A + (static_cast<long long>(a) * p.G * p.R + g * p.R + r) * p.K;
      for (int k = lane; k < p.K; k += 32) h = fmaf(bf2f(x[k]), bf2f(ar[k]), h);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) h += __shfl_xor_sync(0xffffffffu, h, o);
      h *= s;
    }
    if (lane == 0) {
      uint16_t hb;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(hb) : "f"(h));
      p.H[static_cast<long long>(t) * p.G * p.R16 + j] = hb;
    }
  }
}

__global__ void __launch_bounds__(256) multi_y_kernel(const MultiCall p, const float* base) {
  const int t = blockIdx.y;
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= p.N) return;
  const int a = p.slot[t];
  float y = 0.f;
  if (base) y = base[static_cast<long long>(t) * p.N + n];
  else if (p.bias) y = p.bias_f32 ? static_cast<const float*>(p.bias)[n] : bf2f(static_cast<const uint16_t*>(p.bias)[n]);
  if (a >= 0 && a < p.S) {
    const int g = n / (p.N / p.G);
    const uint16_t* b = p.B + (static_cast<long long>(a) * p.N + n) * p.R;
    const uint16_t* h = p.H + static_cast<long long>(t) * p.G * p.R16 + g * p.R16;
    float s = p.scale[a];
    if (p.row_scale) s = __fmul_rn(s, p.row_scale[t]);
    if (__fmul_rn(s, p.request_scale) != 0.f) {
      float d = 0.f;
      for (int r = 0; r < p.R; ++r) d = fmaf(bf2f(h[r]), bf2f(b[r]), d);
      y += d;
    }
  }
  const long long o = static_cast<long long>(t) * p.ldy + n;
  if (p.y_f32) {
    static_cast<float*>(p.Y)[o] = y;
  } else {
    uint16_t yb;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(yb) : "f"(y));
    static_cast<uint16_t*>(p.Y)[o] = yb;
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t r256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int check(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  if (!X || !bank) return WP_ERR_INVALID;
  if (X->rows < 0 || X->cols <= 0 || X->ld < X->cols) return WP_ERR_INVALID;
  if (X->dtype != WP_BF16 || bank->dtype != WP_BF16) return WP_ERR_DTYPE;
  if (bank->n_slots < 1 || bank->n_groups < 1 || bank->rank < 1 || bank->in <= 0 || bank->out <= 0)
    return WP_ERR_INVALID;
  if (bank->n_groups > kMaxGroups || bank->rank > 256) return WP_ERR_UNSUPPORTED;
  if (bank->in != X->cols || bank->out % bank->n_groups) return WP_ERR_SHAPE;
  if (bank->rank % 8) return WP_ERR_SHAPE;
  if (X->cols % 8 || (bank->out / bank->n_groups) % 8) return WP_ERR_ALIGN;
  if (X->rows > 0x7FFFFFFFll || X->cols > 0x7FFFFFFFll || bank->out > 0x7FFFFFFFll) return WP_ERR_UNSUPPORTED;
  if (W) {
    if (W->dtype != WP_BF16 && W->dtype != WP_NF4) return WP_ERR_DTYPE;
    if (W->rows <= 0 || W->cols <= 0 || W->ld < W->cols) return WP_ERR_INVALID;
    if (W->rows != bank->out || W->cols != bank->in) return WP_ERR_SHAPE;
    if (W->dtype == WP_NF4 && (W->cols % 64 || W->ld != W->cols)) return WP_ERR_SHAPE;
  }
  return WP_OK;
}

// Rows up to which the weight-streaming kernels take a bf16 weight (or none).
constexpr int kSmallRows = 512;
bool small_rows(int T, const wp_mat* W) { return T <= kSmallRows && (!W || W->dtype == WP_BF16); }

struct Layout {
  size_t h = 0, act = 0, base = 0, fwd = 0, total = 0;
};

Layout layout(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  Layout L;
  const size_t T = static_cast<size_t>(X->rows);
  const size_t r16 = (bank->rank + 15) / 16 * 16;
  L.act = r256(T * bank->n_groups * r16 * 2);
  L.base = L.act + r256(T * 4);
  L.total = L.fwd = L.base;
  if (W && !small_rows(static_cast<int>(T), W)) {
    L.fwd = L.base + r256(T * bank->out * 4);
    L.total = L.fwd + r256(lora_workspace_size(WP_OP_FWD, X, W, nullptr, 0));
  }
  return L;
}

}  // namespace
}  // namespace wp

using namespace wp;

extern "C" {

size_t lora_multi_workspace_size(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  if (check(X, W, bank) != WP_OK || X->rows == 0) return 0;
  return layout(X, W, bank).total;
}

int lora_linear_fwd_multi(const wp_mat* X, const wp_mat* W, const wp_mat* bias, const wp_bank* bank,
                          const int32_t* slot, const float* row_scale, double request_scale,
                          const wp_out* Y, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check(X, W, bank);
  if (rc != WP_OK) return rc;
  if (!Y || Y->rows < 0 || Y->cols <= 0 || Y->ld < Y->cols || (Y->dtype != WP_BF16 && Y->dtype != WP_FP32))
    return WP_ERR_INVALID;
  if (Y->rows != X->rows || Y->cols != bank->out) return WP_ERR_SHAPE;
  const float rs = static_cast<float>(request_scale);
  if (!std::isfinite(rs)) return WP_ERR_INVALID;
  if (bias) {
    if (!bias->data || (bias->dtype != WP_BF16 && bias->dtype != WP_FP32)) return WP_ERR_INVALID;
    if (bias->rows * bias->cols != bank->out) return WP_ERR_SHAPE;
  }
  if (X->rows == 0) return WP_OK;
  if (!X->data || !Y->data || !bank->A || !bank->B || !bank->scale || !slot) return WP_ERR_INVALID;
  if (W && (!W->data || (W->dtype == WP_NF4 && !W->absmax))) return WP_ERR_INVALID;
  if (!al16(X->data) || X->ld % 8 || !al16(bank->A) || !al16(bank->B)) return WP_ERR_ALIGN;
  if (W && (!al16(W->data) || W->ld % 8)) return WP_ERR_ALIGN;
  if (!al16(Y->data) || Y->ld % (Y->dtype == WP_BF16 ? 8 : 4)) return WP_ERR_ALIGN;
  const Layout L = layout(X, W, bank);
  if (!workspace || workspace_bytes < L.total) return WP_ERR_WORKSPACE;
  if (!al16(workspace)) return WP_ERR_ALIGN;

  char* ws = static_cast<char*>(workspace);
  MultiCall c{};
  c.T = static_cast<int>(X->rows); c.K = static_cast<int>(X->cols); c.N = static_cast<int>(bank->out);
  c.G = bank->n_groups; c.og = c.N / c.G;
  c.R = bank->rank; c.R16 = (c.R + 15) / 16 * 16; c.S = bank->n_slots;
  c.X = static_cast<const uint16_t*>(X->data); c.ldx = X->ld;
  c.A = static_cast<const uint16_t*>(bank->A); c.B = static_cast<const uint16_t*>(bank->B);
  c.scale = bank->scale; c.slot = slot; c.row_scale = row_scale; c.request_scale = rs;
  c.H = reinterpret_cast<uint16_t*>(ws + L.h);
  c.act = reinterpret_cast<int*>(ws + L.act);
  if (bias) {
    c.bias = bias->data;
    c.bias_f32 = bias->dtype == WP_FP32;
  }
  c.Y = Y->data; c.ldy = Y->ld; c.y_f32 = Y->dtype == WP_FP32;
  c.status = tc_status_ptr();
  c.timeout_ns = device_wait_limit_ns();
  if (!c.status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (small_rows(c.T, W)) {
    rc = launch_multi_shrink_small(c, st);
    if (rc != WP_OK) return rc;
    return launch_multi_small(c, W ? W->data : nullptr, W ? W->ld : 0, st);
  }
  const float* base = nullptr;
  if (W) {
    const wp_out by{ws + L.base, WP_FP32, X->rows, bank->out, bank->out};
    rc = lora_linear_fwd(X, W, bias, nullptr, 0, 1.0, &by, ws + L.fwd, L.total - L.fwd, stream);
    if (rc != WP_OK) return rc;
    base = reinterpret_cast<const float*>(ws + L.base);
    c.bias = nullptr;
  }
  multi_h_kernel<<<c.T, 256, 0, st>>>(c);
  for (int t0 = 0; t0 < c.T; t0 += 65535) {
    MultiCall q = c;
    q.T = c.T - t0 < 65535 ? c.T - t0 : 65535;
    q.slot += t0;
    if (q.row_scale) q.row_scale += t0;
    q.H += static_cast<long long>(t0) * c.G * c.R16;
    q.Y = static_cast<char*>(c.Y) + static_cast<long long>(t0) * c.ldy * (c.y_f32 ? 4 : 2);
    multi_y_kernel<<<dim3((c.N + 255) / 256, q.T), 256, 0, st>>>(
        q, base ? base + static_cast<long long>(t0) * c.N : nullptr);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return WP_ERR_CUDA;
  }
  return WP_OK;
}

}  // extern "C"
