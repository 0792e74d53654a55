// wp_norm.cu -- layer norm and the form without a mean, forward and backward.
//
//   forward   y = (x - mu) r w + b,  r = 1 / sqrt(var + eps)
//   backward  xh = (x - mu) r, h = dy w
//             dx = r (h - mean(h) - xh mean(h xh))       (no mean(h) without a mean)
//             dw = sum_t dy xh,  db = sum_t dy
//
// Both are bound by HBM: a row is read once into registers, its sums are taken there (the
// squares after the mean is out, so that a large mean costs no digits), and written once.
// TPR threads share a row; a CTA of 256 or more threads holds several short rows at a time
// or one long one.  The backward keeps a CTA on its rows' columns: every thread owns the
// same columns of each row it meets, so the column sums dw and db stay in registers over all
// of the CTA's rows, are joined in the CTA in a fixed order, and one partial row per CTA goes
// to the workspace, which a second kernel adds in order: no atomics, the same bits each time.
#include <cmath>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

struct NormParams {
  long long T;
  int C;
  const void* x; long long ldx;
  const void* dy; long long lddy;
  const void* w; int w_f32;
  const void* b; int b_f32;
  void* y; long long ldy;          // forward: y; backward: dx (may be null)
  float* stats;                    // [2, T]: written (may be null) / read
  float eps;
  float inv_c;
  float* part;                     // backward: [gridDim.x][2][C] partial dw, db (may be null)
};

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }

// V consecutive elements of a row as fp32
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) v[0] = bf2f(__ldg(reinterpret_cast<const unsigned short*>(p)));
    else v[0] = __ldg(reinterpret_cast<const float*>(p));
  } else {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf2f(u[k] & 0xffffu);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(u[k]);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) {
      uint16_t h;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v[0]));
      *reinterpret_cast<uint16_t*>(p) = h;
    } else {
      *reinterpret_cast<float*>(p) = v[0];
    }
  } else if constexpr (sizeof(T) == 2) {
    st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7]));
  } else {
    st_global_v4(p, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
}

__device__ __forceinline__ float vec_at(const void* p, int f32, int c) {
  return f32 ? __ldg(static_cast<const float*>(p) + c) : bf2f(__ldg(static_cast<const unsigned short*>(p) + c));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the TPR threads that share a row; `red` has one entry per warp of the CTA and is
// not used by the row's previous sum (the callers alternate two).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int first = threadIdx.x / TPR * (TPR / 32);
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[first + i];
  }
  return v;
}

constexpr int kNormThreads = 256;

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads)
    norm_fwd_kernel(const NormParams p, const bool layer) {
  constexpr int kThreads = TPR > kNormThreads ? TPR : kNormThreads;
  constexpr int kRows = kThreads / TPR;
  __shared__ float red[2][kThreads / 32];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  for (long long base = static_cast<long long>(blockIdx.x) * kRows; base < p.T;
       base += static_cast<long long>(gridDim.x) * kRows) {
    const long long row = base + sub;
    const bool ok = row < p.T;
    const T* xr = static_cast<const T*>(p.x) + (ok ? row : 0) * p.ldx;
    float x[NV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c < p.C) {
        load_row<T, V>(xr + c, x[i]);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) x[i][k] = 0.f;
      }
    }
    float mu = 0.f;
    if (layer) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) s += x[i][k];
      mu = row_sum<TPR>(s, red[0]) * p.inv_c;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i * TPR + lane) * V < p.C) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float d = x[i][k] - mu;
          ss = fmaf(d, d, ss);
        }
      }
    }
    const float r = 1.0f / sqrtf(row_sum<TPR>(ss, red[1]) * p.inv_c + p.eps);
    if (ok) {
      if (p.stats && lane == 0) {
        p.stats[row] = mu;
        p.stats[p.T + row] = r;
      }
      T* yr = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (c < p.C) {
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) {
            o[k] = (x[i][k] - mu) * r;
            if (p.w) o[k] *= vec_at(p.w, p.w_f32, c + k);
            if (p.b) o[k] += vec_at(p.b, p.b_f32, c + k);
          }
          store_row<T, V>(yr + c, o);
        }
      }
    }
    if (TPR > 32 && !layer) __syncthreads();   // red[1] of this row is read before the next row's sum
  }
}

// Rows too long for the registers of 512 threads: three passes over the row.
template <typename T>
__global__ void __launch_bounds__(512) norm_fwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[2][16];
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    float mu = 0.f, v[1];
    if (layer) {
      float s = 0.f;
      for (int c = threadIdx.x; c < p.C; c += 512) {
        load_row<T, 1>(xr + c, v);
        s += v[0];
      }
      mu = row_sum<512>(s, red[0]) * p.inv_c;
    }
    float ss = 0.f;
    for (int c = threadIdx.x; c < p.C; c += 512) {
      load_row<T, 1>(xr + c, v);
      ss = fmaf(v[0] - mu, v[0] - mu, ss);
    }
    const float r = 1.0f / sqrtf(row_sum<512>(ss, red[1]) * p.inv_c + p.eps);
    if (p.stats && threadIdx.x == 0) {
      p.stats[row] = mu;
      p.stats[p.T + row] = r;
    }
    T* yr = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x; c < p.C; c += 512) {
      load_row<T, 1>(xr + c, v);
      v[0] = (v[0] - mu) * r;
      if (p.w) v[0] *= vec_at(p.w, p.w_f32, c);
      if (p.b) v[0] += vec_at(p.b, p.b_f32, c);
      store_row<T, 1>(yr + c, v);
    }
    __syncthreads();
  }
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(TPR > kNormThreads ? TPR : kNormThreads)
    norm_bwd_kernel(const NormParams p, const bool layer) {
  constexpr int kThreads = TPR > kNormThreads ? TPR : kNormThreads;
  constexpr int kRows = kThreads / TPR;
  __shared__ float red[2][2][kThreads / 32];
  extern __shared__ float colsum[];            // [kRows - 1 > 0 ? kRows : 0][C] of one of dw, db
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.f;
  int turn = 0;
  for (long long base = static_cast<long long>(blockIdx.x) * kRows; base < p.T;
       base += static_cast<long long>(gridDim.x) * kRows, turn ^= 1) {
    const long long row = base + sub;
    const bool ok = row < p.T;
    const T* xr = static_cast<const T*>(p.x) + (ok ? row : 0) * p.ldx;
    const T* gr = static_cast<const T*>(p.dy) + (ok ? row : 0) * p.lddy;
    const float mu = layer && ok ? p.stats[row] : 0.f;
    const float r = ok ? p.stats[p.T + row] : 0.f;
    float x[NV][V], g[NV][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (ok && c < p.C) {
        load_row<T, V>(xr + c, x[i]);
        load_row<T, V>(gr + c, g[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * V;
      if (ok && c < p.C) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          x[i][k] = (x[i][k] - mu) * r;
          dw[i][k] = fmaf(g[i][k], x[i][k], dw[i][k]);
          db[i][k] += g[i][k];
          if (p.w) g[i][k] *= vec_at(p.w, p.w_f32, c + k);
          s1 += g[i][k];
          s2 = fmaf(g[i][k], x[i][k], s2);
        }
      }
    }
    if (p.y) {
      const float m1 = layer ? row_sum<TPR>(s1, red[turn][0]) * p.inv_c : 0.f;
      const float m2 = row_sum<TPR>(s2, red[turn][1]) * p.inv_c;
      T* yr = static_cast<T*>(p.y) + (ok ? row : 0) * p.ldy;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
        if (ok && c < p.C) {
          float o[V];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = r * (g[i][k] - m1 - x[i][k] * m2);
          store_row<T, V>(yr + c, o);
        }
      }
    }
  }
  if (!p.part) return;
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.C;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (kRows == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * V;
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c + k < p.C) out[which * p.C + c + k] = which ? db[i][k] : dw[i][k];
      }
    } else {
      // the rows' threads take turns adding into one row of shared memory, in order
      for (int s = 0; s < kRows; ++s) {
        if (sub == s) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + lane) * V;
#pragma unroll
            for (int k = 0; k < V; ++k)
              if (c + k < p.C) {
                const float a = which ? db[i][k] : dw[i][k];
                colsum[c + k] = s == 0 ? a : colsum[c + k] + a;
              }
          }
        }
        __syncthreads();
      }
      for (int c = threadIdx.x; c < p.C; c += kThreads) out[which * p.C + c] = colsum[c];
      __syncthreads();
    }
  }
}

// Rows too long for registers: sums of a row from two passes; a thread's columns are strided
// by 512, its dw and db kept in the CTA's own workspace row (each element touched by one
// thread only).
template <typename T>
__global__ void __launch_bounds__(512) norm_bwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[2][16];
  float* out = p.part ? p.part + static_cast<long long>(blockIdx.x) * 2 * p.C : nullptr;
  if (out)
    for (int c = threadIdx.x; c < p.C; c += 512) out[c] = out[p.C + c] = 0.f;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    const T* gr = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mu = layer ? p.stats[row] : 0.f, r = p.stats[p.T + row];
    float xv[1], gv[1], s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < p.C; c += 512) {
      load_row<T, 1>(xr + c, xv);
      load_row<T, 1>(gr + c, gv);
      const float xh = (xv[0] - mu) * r;
      if (out) {
        out[c] = fmaf(gv[0], xh, out[c]);
        out[p.C + c] += gv[0];
      }
      const float h = p.w ? gv[0] * vec_at(p.w, p.w_f32, c) : gv[0];
      s1 += h;
      s2 = fmaf(h, xh, s2);
    }
    if (p.y) {
      const float m1 = layer ? row_sum<512>(s1, red[0]) * p.inv_c : 0.f;
      const float m2 = row_sum<512>(s2, red[1]) * p.inv_c;
      T* yr = static_cast<T*>(p.y) + row * p.ldy;
      for (int c = threadIdx.x; c < p.C; c += 512) {
        load_row<T, 1>(xr + c, xv);
        load_row<T, 1>(gr + c, gv);
        const float xh = (xv[0] - mu) * r;
        const float h = p.w ? gv[0] * vec_at(p.w, p.w_f32, c) : gv[0];
        float o[1] = {r * (h - m1 - xh * m2)};
        store_row<T, 1>(yr + c, o);
      }
      __syncthreads();
    }
  }
}

// dw, db [C] from the CTAs' partial rows: 32 columns a block, 8 warps take every eighth
// partial row, joined in warp order.
__global__ void __launch_bounds__(256) norm_finish_kernel(const float* part, int n, int C, float* dw, float* db) {
  __shared__ float sh[8][33];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  float s = 0.f;
  if (c < C)
    for (int i = warp; i < n; i += 8) s += part[(static_cast<long long>(i) * 2 + blockIdx.y) * C + c];
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < C) {
    float t = sh[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sh[i][lane];
    out[c] = t;
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int last_launch() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

bool valid_vec(const wp_mat* v, long long C) {
  return v->data && (v->dtype == WP_BF16 || v->dtype == WP_FP32) && v->rows >= 1 && v->cols >= 1 &&
         v->rows * v->cols == C;
}

// CTAs of the backward: each carries its columns' sums, so more CTAs mean more partial rows
int bwd_grid(long long T, int rows_per_cta) {
  const long long need = (T + rows_per_cta - 1) / rows_per_cta;
  const long long cap = 2ll * device_sm_count();
  return static_cast<int>(need < cap ? need : cap);
}

template <typename T, int V, int NV, int TPR>
int run_fwd(const NormParams& p, bool layer, cudaStream_t st) {
  constexpr int kThreads = TPR > kNormThreads ? TPR : kNormThreads;
  const long long need = (p.T + kThreads / TPR - 1) / (kThreads / TPR);
  const long long cap = 1ll << 20;
  norm_fwd_kernel<T, V, NV, TPR><<<static_cast<unsigned>(need < cap ? need : cap), kThreads, 0, st>>>(p, layer);
  return last_launch();
}

template <typename T, int V, int NV, int TPR>
int run_bwd(const NormParams& p, bool layer, int* grid, cudaStream_t st) {
  constexpr int kThreads = TPR > kNormThreads ? TPR : kNormThreads;
  constexpr int kRows = kThreads / TPR;
  *grid = bwd_grid(p.T, kRows);
  const size_t smem = kRows > 1 ? static_cast<size_t>(p.C) * 4 : 0;
  norm_bwd_kernel<T, V, NV, TPR><<<*grid, kThreads, smem, st>>>(p, layer);
  return last_launch();
}

template <typename T>
int dispatch_fwd(const NormParams& p, bool vec, bool layer, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    const int nv = p.C / V;
    if (nv <= 32 * 8) return run_fwd<T, V, 8, 32>(p, layer, st);
    if (nv <= 256 * 4) return run_fwd<T, V, 4, 256>(p, layer, st);
    if (nv <= 512 * 8) return run_fwd<T, V, 8, 512>(p, layer, st);
  } else {
    if (p.C <= 32 * 16) return run_fwd<T, 1, 16, 32>(p, layer, st);
    if (p.C <= 256 * 32) return run_fwd<T, 1, 32, 256>(p, layer, st);
    if (p.C <= 512 * 32) return run_fwd<T, 1, 32, 512>(p, layer, st);
  }
  norm_fwd_long_kernel<T><<<static_cast<unsigned>(p.T < (1 << 20) ? p.T : (1 << 20)), 512, 0, st>>>(p, layer);
  return last_launch();
}

template <typename T>
int dispatch_bwd(const NormParams& p, bool vec, bool layer, int* grid, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    const int nv = p.C / V;
    if (nv <= 32 * 6) return run_bwd<T, V, 6, 32>(p, layer, grid, st);
    if (nv <= 256 * 4) return run_bwd<T, V, 4, 256>(p, layer, grid, st);
    if (nv <= 512 * 4) return run_bwd<T, V, 4, 512>(p, layer, grid, st);
  } else {
    if (p.C <= 32 * 16) return run_bwd<T, 1, 16, 32>(p, layer, grid, st);
    if (p.C <= 256 * 20) return run_bwd<T, 1, 20, 256>(p, layer, grid, st);
    if (p.C <= 512 * 28) return run_bwd<T, 1, 28, 512>(p, layer, grid, st);
  }
  *grid = bwd_grid(p.T, 1);
  norm_bwd_long_kernel<T><<<*grid, 512, 0, st>>>(p, layer);
  return last_launch();
}

bool valid_rows(const wp_mat* m) {
  return m && m->rows >= 0 && m->cols > 0 && (m->data || m->rows == 0) && m->ld >= m->cols &&
         (m->dtype == WP_BF16 || m->dtype == WP_FP32);
}

}  // namespace

size_t norm_bwd_workspace(long long T, long long C) {
  // a partial row of dw and db for each CTA of the backward
  if (T < 0 || C <= 0) return 0;
  const long long n = T < 2ll * device_sm_count() ? T : 2ll * device_sm_count();
  return (static_cast<size_t>(n) * 2 * C * 4 + 255) & ~static_cast<size_t>(255);
}

}  // namespace wp

using namespace wp;

extern "C" {

int lora_norm_fwd(const wp_mat* X, const wp_mat* weight, const wp_mat* bias, int32_t kind, double eps,
                  const wp_out* Y, float* stats, void* stream) {
  if (!valid_rows(X) || !Y || Y->rows < 0 || Y->cols <= 0 || Y->ld < Y->cols || (!Y->data && Y->rows != 0))
    return WP_ERR_INVALID;
  if (kind != WP_NORM_LAYER && kind != WP_NORM_RMS) return WP_ERR_INVALID;
  if (!std::isfinite(eps) || eps < 0) return WP_ERR_INVALID;
  if (Y->dtype != X->dtype) return WP_ERR_DTYPE;
  if (Y->rows != X->rows || Y->cols != X->cols) return WP_ERR_SHAPE;
  if (weight && !valid_vec(weight, X->cols)) return weight->data ? WP_ERR_SHAPE : WP_ERR_INVALID;
  if (bias && !valid_vec(bias, X->cols)) return bias->data ? WP_ERR_SHAPE : WP_ERR_INVALID;
  if (X->cols > 0x3FFFFFFFLL) return WP_ERR_UNSUPPORTED;
  if (X->rows == 0) return WP_OK;
  NormParams p{};
  p.T = X->rows; p.C = static_cast<int>(X->cols);
  p.x = X->data; p.ldx = X->ld;
  p.w = weight ? weight->data : nullptr; p.w_f32 = weight && weight->dtype == WP_FP32;
  p.b = bias ? bias->data : nullptr; p.b_f32 = bias && bias->dtype == WP_FP32;
  p.y = Y->data; p.ldy = Y->ld;
  p.stats = stats;
  p.eps = static_cast<float>(eps);
  p.inv_c = 1.0f / static_cast<float>(p.C);
  const int V = X->dtype == WP_BF16 ? 8 : 4;
  const bool vec = p.C % V == 0 && p.ldx % V == 0 && p.ldy % V == 0 && al16(p.x) && al16(p.y);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool layer = kind == WP_NORM_LAYER;
  return X->dtype == WP_BF16 ? dispatch_fwd<uint16_t>(p, vec, layer, st) : dispatch_fwd<float>(p, vec, layer, st);
}

int lora_norm_bwd(const wp_mat* dY, const wp_mat* X, const wp_mat* weight, const float* stats, int32_t kind,
                  const wp_out* dX, const wp_out* dW, const wp_out* dB, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (!valid_rows(X) || !valid_rows(dY)) return WP_ERR_INVALID;
  if (kind != WP_NORM_LAYER && kind != WP_NORM_RMS) return WP_ERR_INVALID;
  if (!stats && X->rows != 0) return WP_ERR_INVALID;
  if (dX && (dX->rows < 0 || dX->cols <= 0 || dX->ld < dX->cols || (!dX->data && dX->rows != 0))) return WP_ERR_INVALID;
  if (dY->dtype != X->dtype || (dX && dX->dtype != X->dtype)) return WP_ERR_DTYPE;
  if (dY->rows != X->rows || dY->cols != X->cols) return WP_ERR_SHAPE;
  if (dX && (dX->rows != X->rows || dX->cols != X->cols)) return WP_ERR_SHAPE;
  if (weight && !valid_vec(weight, X->cols)) return weight->data ? WP_ERR_SHAPE : WP_ERR_INVALID;
  for (const wp_out* o : {dW, dB}) {
    if (!o) continue;
    if (!o->data) return WP_ERR_INVALID;
    if (o->dtype != WP_FP32) return WP_ERR_DTYPE;
    if (o->rows * o->cols != X->cols) return WP_ERR_SHAPE;
  }
  if (X->cols > 0x3FFFFFFFLL) return WP_ERR_UNSUPPORTED;
  const bool sums = dW || dB;
  const size_t need = sums ? norm_bwd_workspace(X->rows, X->cols) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need)) return WP_ERR_WORKSPACE;
  if (need > 0 && !al16(workspace)) return WP_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (X->rows == 0) {
    for (const wp_out* o : {dW, dB}) {
      if (!o) continue;
      const cudaError_t e = cudaMemsetAsync(o->data, 0, static_cast<size_t>(X->cols) * 4, st);
      if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return WP_ERR_CUDA;
      }
    }
    return WP_OK;
  }
  if (!sums && !dX) return WP_OK;
  NormParams p{};
  p.T = X->rows; p.C = static_cast<int>(X->cols);
  p.x = X->data; p.ldx = X->ld;
  p.dy = dY->data; p.lddy = dY->ld;
  p.w = weight ? weight->data : nullptr; p.w_f32 = weight && weight->dtype == WP_FP32;
  p.y = dX ? dX->data : nullptr; p.ldy = dX ? dX->ld : 0;
  p.stats = const_cast<float*>(stats);
  p.inv_c = 1.0f / static_cast<float>(p.C);
  p.part = sums ? static_cast<float*>(workspace) : nullptr;
  const int V = X->dtype == WP_BF16 ? 8 : 4;
  const bool vec = p.C % V == 0 && p.ldx % V == 0 && p.lddy % V == 0 && al16(p.x) && al16(p.dy) &&
                   (!dX || (p.ldy % V == 0 && al16(p.y)));
  const bool layer = kind == WP_NORM_LAYER;
  int grid = 0;
  const int rc = X->dtype == WP_BF16 ? dispatch_bwd<uint16_t>(p, vec, layer, &grid, st)
                                     : dispatch_bwd<float>(p, vec, layer, &grid, st);
  if (rc != WP_OK || !sums) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.C + 31) / 32, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_finish_kernel, static_cast<const float*>(p.part), grid, p.C,
                                           dW ? static_cast<float*>(dW->data) : nullptr,
                                           dB ? static_cast<float*>(dB->data) : nullptr);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return WP_ERR_CUDA;
  }
  return WP_OK;
}

}  // extern "C"
