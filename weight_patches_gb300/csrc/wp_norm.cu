// wp_norm.cu -- layer norm and the form without a mean, forward and backward.
//
//   forward   y = (x - mu) r w + b,  r = 1 / sqrt(var + eps)
//   backward  xh = (x - mu) r, h = dy w
//             dx = r (h - mean(h) - xh mean(h xh))       (no mean(h) without a mean)
//             dw = sum_t dy xh,  db = sum_t dy
//
// Both are bound by HBM: a row is read once into registers (kept as loaded, unpacked at each
// use), its sums are taken there (the squares after the mean is out, so that a large mean costs
// no digits), and written once.  Forward: short rows a warp each, longer ones a CTA each.
// Backward: a CTA's threads keep their columns over all of its rows, so the column sums dw and db
// stay in registers; it takes several rows per turn where a thread has few columns, so that one
// barrier serves them all and enough loads are in flight.  Each CTA leaves one partial row of dw
// and db in the workspace, which a second kernel adds in order: no atomics, the same bits each
// time.
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
  const void* w; int w_f32, w_vec;   // _vec: 16-byte loads of V columns are aligned
  const void* b; int b_f32, b_vec;
  void* y; long long ldy;          // forward: y; backward: dx (may be null)
  float* stats;                    // [2, T]: written (may be null) / read
  float eps;
  float inv_c;
  float* part;                     // backward: [gridDim.x][2][C] partial dw, db (may be null)
};

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }

// V consecutive elements of a row as loaded
template <typename T, int V>
struct Raw {
  uint32_t u[V * sizeof(T) < 4 ? 1 : V * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V > 1) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
      u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
    } else if constexpr (sizeof(T) == 2) {
      u[0] = static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16;
    } else {
      u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& w : u) w = 0;
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (sizeof(T) == 4 || V == 1) return __uint_as_float(u[k]);
    return __uint_as_float(k & 1 ? u[k >> 1] & 0xffff0000u : u[k >> 1] << 16);
  }
};

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

// V values of a weight or bias vector (either type) from column c, 16 bytes at a time where the
// vector's base allows (the rows' V columns start at multiples of V)
template <int V>
__device__ __forceinline__ void load_vec(const void* p, int f32, int vec, int c, float (&v)[V]) {
  if (V > 1 && vec) {
    if (f32) {
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + k));
        v[k] = q.x; v[k + 1] = q.y; v[k + 2] = q.z; v[k + 3] = q.w;
      }
      return;
    }
    if constexpr (V == 8) {
      Raw<uint16_t, 8> r;
      r.load(static_cast<const uint16_t*>(p) + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = r.at(k);
      return;
    }
    if constexpr (V == 4) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + c));
      v[0] = bf2f(q.x & 0xffffu); v[1] = __uint_as_float(q.x & 0xffff0000u);
      v[2] = bf2f(q.y & 0xffffu); v[3] = __uint_as_float(q.y & 0xffff0000u);
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    v[k] = f32 ? __ldg(static_cast<const float*>(p) + c + k) : bf2f(__ldg(static_cast<const unsigned short*>(p) + c + k));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over the CTA: red holds N per warp and is not used by the sum before (the
// callers alternate two).
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* red) {
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[(threadIdx.x >> 5) * N + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += red[w * N + i];
}

constexpr int kMaxThreads = 512;

// One row: its raw elements in x, thread `lane` of `tpr` holding vectors lane, lane + tpr, ...
template <typename T, int V, int NV, bool kWarp>
__device__ __forceinline__ void fwd_row(const NormParams& p, bool layer, long long row, int lane, int tpr, float* red) {
  const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
  Raw<T, V> x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
    if (c < p.C) x[i].load(xr + c);
    else x[i].zero();
  }
  float mu = 0.f;
  if (layer) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) s[0] += x[i].at(k);
    if constexpr (kWarp) s[0] = warp_sum(s[0]);
    else cta_sum<1>(s, red);
    mu = s[0] * p.inv_c;
  }
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * tpr + lane) * V < p.C)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float d = x[i].at(k) - mu;
        ss[0] = fmaf(d, d, ss[0]);
      }
  if constexpr (kWarp) ss[0] = warp_sum(ss[0]);
  else cta_sum<1>(ss, red + 32);
  const float r = 1.0f / sqrtf(ss[0] * p.inv_c + p.eps);
  if (p.stats && lane == 0) {
    p.stats[row] = mu;
    p.stats[p.T + row] = r;
  }
  T* yr = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
    if (c < p.C) {
      float o[V], q[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = (x[i].at(k) - mu) * r;
      if (p.w) {
        load_vec<V>(p.w, p.w_f32, p.w_vec, c, q);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] *= q[k];
      }
      if (p.b) {
        load_vec<V>(p.b, p.b_f32, p.b_vec, c, q);
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] += q[k];
      }
      store_row<T, V>(yr + c, o);
    }
  }
}

// Short rows: a warp each, 8 warps per CTA.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(256) norm_fwd_warp_kernel(const NormParams p, const bool layer) {
  const long long stride = static_cast<long long>(gridDim.x) * 8;
  for (long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < p.T; row += stride)
    fwd_row<T, V, NV, true>(p, layer, row, threadIdx.x & 31, 32, nullptr);
}

// Longer rows: a CTA each.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_cta_kernel(const NormParams p, const bool layer) {
  __shared__ float red[64];
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    fwd_row<T, V, NV, false>(p, layer, row, threadIdx.x, blockDim.x, red);
    __syncthreads();                     // the sums are read before the next row's are written
  }
}

// Rows too long for the registers of 512 threads: three passes over the row.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[64];
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    float mu = 0.f;
    Raw<T, 1> v;
    if (layer) {
      float s[1] = {0.f};
      for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
        v.load(xr + c);
        s[0] += v.at(0);
      }
      cta_sum<1>(s, red);
      mu = s[0] * p.inv_c;
    }
    float ss[1] = {0.f};
    for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
      v.load(xr + c);
      ss[0] = fmaf(v.at(0) - mu, v.at(0) - mu, ss[0]);
    }
    cta_sum<1>(ss, red + 32);
    const float r = 1.0f / sqrtf(ss[0] * p.inv_c + p.eps);
    if (p.stats && threadIdx.x == 0) {
      p.stats[row] = mu;
      p.stats[p.T + row] = r;
    }
    T* yr = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
      v.load(xr + c);
      float o[1] = {(v.at(0) - mu) * r}, q[1];
      if (p.w) {
        load_vec<1>(p.w, p.w_f32, 0, c, q);
        o[0] *= q[0];
      }
      if (p.b) {
        load_vec<1>(p.b, p.b_f32, 0, c, q);
        o[0] += q[0];
      }
      store_row<T, 1>(yr + c, o);
    }
    __syncthreads();
  }
}

// ROWS rows of a CTA per turn: thread t holds vectors t, t + blockDim, ... of each.
template <typename T, int V, int NV, int ROWS>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const NormParams p, const bool layer) {
  __shared__ float red[2][16 * 2 * ROWS];
  const int lane = threadIdx.x, tpr = blockDim.x;
  float dw[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dw[i][k] = db[i][k] = 0.f;
  int turn = 0;
  for (long long row0 = static_cast<long long>(blockIdx.x) * ROWS; row0 < p.T;
       row0 += static_cast<long long>(gridDim.x) * ROWS, turn ^= 1) {
    Raw<T, V> x[ROWS][NV], g[ROWS][NV];
    float mu[ROWS], r[ROWS], s[2 * ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const long long row = row0 + j;
      const bool ok = row < p.T;
      const T* xr = static_cast<const T*>(p.x) + (ok ? row : 0) * p.ldx;
      const T* gr = static_cast<const T*>(p.dy) + (ok ? row : 0) * p.lddy;
      mu[j] = layer && ok ? __ldg(p.stats + row) : 0.f;
      r[j] = ok ? __ldg(p.stats + p.T + row) : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * V;
        if (ok && c < p.C) {
          x[j][i].load(xr + c);
          g[j][i].load(gr + c);
        } else {
          x[j][i].zero();
          g[j][i].zero();
        }
      }
    }
    float w[V];
#pragma unroll
    for (int k = 0; k < 2 * ROWS; ++k) s[k] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * tpr + lane) * V;
      if (c < p.C) {
        if (p.w) load_vec<V>(p.w, p.w_f32, p.w_vec, c, w);
#pragma unroll
        for (int j = 0; j < ROWS; ++j)
          if (row0 + j < p.T)
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const float xh = (x[j][i].at(k) - mu[j]) * r[j], gk = g[j][i].at(k);
              dw[i][k] = fmaf(gk, xh, dw[i][k]);
              db[i][k] += gk;
              const float h = p.w ? gk * w[k] : gk;
              s[2 * j] += h;
              s[2 * j + 1] = fmaf(h, xh, s[2 * j + 1]);
            }
      }
    }
    if (p.y) {
      cta_sum<2 * ROWS>(s, red[turn]);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * tpr + lane) * V;
        if (c < p.C) {
          if (p.w) load_vec<V>(p.w, p.w_f32, p.w_vec, c, w);
#pragma unroll
          for (int j = 0; j < ROWS; ++j)
            if (row0 + j < p.T) {
              const float m1 = layer ? s[2 * j] * p.inv_c : 0.f, m2 = s[2 * j + 1] * p.inv_c;
              float o[V];
#pragma unroll
              for (int k = 0; k < V; ++k) {
                const float xh = (x[j][i].at(k) - mu[j]) * r[j];
                const float h = p.w ? g[j][i].at(k) * w[k] : g[j][i].at(k);
                o[k] = r[j] * (h - m1 - xh * m2);
              }
              store_row<T, V>(static_cast<T*>(p.y) + (row0 + j) * p.ldy + c, o);
            }
        }
      }
    }
  }
  if (!p.part) return;
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.C;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * tpr + lane) * V;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (c + k < p.C) {
        out[c + k] = dw[i][k];
        out[p.C + c + k] = db[i][k];
      }
  }
}

// Rows too long for registers: sums of a row from two passes; a thread's columns are strided
// by 512, its dw and db kept in the CTA's own workspace row (each element touched by one
// thread only).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[32];
  float* out = p.part ? p.part + static_cast<long long>(blockIdx.x) * 2 * p.C : nullptr;
  if (out)
    for (int c = threadIdx.x; c < p.C; c += kMaxThreads) out[c] = out[p.C + c] = 0.f;
  for (long long row = blockIdx.x; row < p.T; row += gridDim.x) {
    const T* xr = static_cast<const T*>(p.x) + row * p.ldx;
    const T* gr = static_cast<const T*>(p.dy) + row * p.lddy;
    const float mu = layer ? p.stats[row] : 0.f, r = p.stats[p.T + row];
    Raw<T, 1> xv, gv;
    float s[2] = {0.f, 0.f}, w[1] = {1.f};
    for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
      xv.load(xr + c);
      gv.load(gr + c);
      const float xh = (xv.at(0) - mu) * r;
      if (out) {
        out[c] = fmaf(gv.at(0), xh, out[c]);
        out[p.C + c] += gv.at(0);
      }
      if (p.w) load_vec<1>(p.w, p.w_f32, 0, c, w);
      const float h = gv.at(0) * w[0];
      s[0] += h;
      s[1] = fmaf(h, xh, s[1]);
    }
    if (p.y) {
      cta_sum<2>(s, red);
      const float m1 = layer ? s[0] * p.inv_c : 0.f, m2 = s[1] * p.inv_c;
      T* yr = static_cast<T*>(p.y) + row * p.ldy;
      for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
        xv.load(xr + c);
        gv.load(gr + c);
        const float xh = (xv.at(0) - mu) * r;
        if (p.w) load_vec<1>(p.w, p.w_f32, 0, c, w);
        float o[1] = {r * (gv.at(0) * w[0] - m1 - xh * m2)};
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

// Threads that share a row: each holds nv vectors of it, a whole number of warps in all.
int row_threads(long long vectors, int nv) {
  return static_cast<int>(((vectors + nv - 1) / nv + 31) / 32 * 32);
}

// Form of the backward for rows of C elements: vectors per thread, rows per turn (four where a
// thread has one vector of each, two for two; the single-element form likewise by elements),
// threads, and the most CTAs (about 1024 threads' worth per SM, two at least: each leaves a partial
// row).  nv 0: the long form.
struct BwdForm {
  int nv, rows, threads, ctas;
};

BwdForm bwd_form(long long C, bool f32, bool vec) {
  const int V = vec ? (f32 ? 4 : 8) : 1;
  const long long n = C / V;
  BwdForm f{0, 1, 512, 0};
  if (vec) {
    if (n <= 320) f = {1, 4, 0, 0};
    else if (n <= 384 * 2) f = {2, 2, 0, 0};
    else if (n <= 512 * 4) f = {4, 1, 0, 0};
  } else {
    if (n <= 256 * 2) f = {2, 4, 0, 0};
    else if (n <= 384 * 8) f = {8, 2, 0, 0};
    else if (n <= 512 * 16) f = {16, 1, 0, 0};
    else if (n <= 512 * 28) f = {28, 1, 0, 0};
  }
  if (f.nv) f.threads = row_threads(n, f.nv);
  const int per_sm = 1024 / f.threads;
  f.ctas = (per_sm < 2 ? 2 : (per_sm > 8 ? 8 : per_sm)) * device_sm_count();
  return f;
}

template <typename T, int V, int NV>
int run_fwd(const NormParams& p, bool layer, cudaStream_t st) {
  const int threads = row_threads(p.C / V, NV);
  norm_fwd_cta_kernel<T, V, NV><<<static_cast<unsigned>(p.T < (1 << 30) ? p.T : (1 << 30)), threads, 0, st>>>(p, layer);
  return last_launch();
}

template <typename T, int V, int NV>
int run_fwd_warp(const NormParams& p, bool layer, cudaStream_t st) {
  const long long need = (p.T + 7) / 8;
  norm_fwd_warp_kernel<T, V, NV><<<static_cast<unsigned>(need < (1 << 30) ? need : (1 << 30)), 256, 0, st>>>(p, layer);
  return last_launch();
}

template <typename T, int V, int NV, int ROWS>
void run_bwd(const NormParams& p, const BwdForm& f, bool layer, int* grid, cudaStream_t st) {
  const long long need = (p.T + ROWS - 1) / ROWS;
  *grid = static_cast<int>(need < f.ctas ? need : f.ctas);
  norm_bwd_kernel<T, V, NV, ROWS><<<*grid, f.threads, 0, st>>>(p, layer);
}

// Short rows take a warp each (no barrier); beyond 8 vectors (16 single elements) a lane, a CTA
// with as few vectors a thread as 256 threads allow.
template <typename T>
int dispatch_fwd(const NormParams& p, bool vec, bool layer, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    const int n = p.C / V;
    if (n <= 32) return run_fwd_warp<T, V, 1>(p, layer, st);
    if (n <= 32 * 4) return run_fwd_warp<T, V, 4>(p, layer, st);
    if (n <= 32 * 8) return run_fwd_warp<T, V, 8>(p, layer, st);
    if (n <= 256 * 2) return run_fwd<T, V, 2>(p, layer, st);
    if (n <= 256 * 4) return run_fwd<T, V, 4>(p, layer, st);
    if (n <= 512 * 8) return run_fwd<T, V, 8>(p, layer, st);
  } else {
    if (p.C <= 32 * 4) return run_fwd_warp<T, 1, 4>(p, layer, st);
    if (p.C <= 32 * 16) return run_fwd_warp<T, 1, 16>(p, layer, st);
    if (p.C <= 256 * 8) return run_fwd<T, 1, 8>(p, layer, st);
    if (p.C <= 512 * 16) return run_fwd<T, 1, 16>(p, layer, st);
    if (p.C <= 512 * 32) return run_fwd<T, 1, 32>(p, layer, st);
  }
  norm_fwd_long_kernel<T><<<static_cast<unsigned>(p.T < (1 << 30) ? p.T : (1 << 30)), kMaxThreads, 0, st>>>(p, layer);
  return last_launch();
}

template <typename T>
int dispatch_bwd(const NormParams& p, bool vec, bool layer, int* grid, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const BwdForm f = bwd_form(p.C, sizeof(T) == 4, vec);
  if (f.nv == 0) {
    *grid = static_cast<int>(p.T < f.ctas ? p.T : f.ctas);
    norm_bwd_long_kernel<T><<<*grid, kMaxThreads, 0, st>>>(p, layer);
  } else if (vec) {
    if (f.nv == 1) run_bwd<T, V, 1, 4>(p, f, layer, grid, st);
    else if (f.nv == 2) run_bwd<T, V, 2, 2>(p, f, layer, grid, st);
    else run_bwd<T, V, 4, 1>(p, f, layer, grid, st);
  } else {
    if (f.nv == 2) run_bwd<T, 1, 2, 4>(p, f, layer, grid, st);
    else if (f.nv == 8) run_bwd<T, 1, 8, 2>(p, f, layer, grid, st);
    else if (f.nv == 16) run_bwd<T, 1, 16, 1>(p, f, layer, grid, st);
    else run_bwd<T, 1, 28, 1>(p, f, layer, grid, st);
  }
  return last_launch();
}

bool valid_rows(const wp_mat* m) {
  return m && m->rows >= 0 && m->cols > 0 && (m->data || m->rows == 0) && m->ld >= m->cols &&
         (m->dtype == WP_BF16 || m->dtype == WP_FP32);
}

}  // namespace

size_t norm_bwd_workspace(long long T, long long C, bool f32) {
  // a partial row of dw and db for each CTA of either form (16-byte aligned rows or not)
  if (T < 0 || C <= 0) return 0;
  long long n = bwd_form(C, f32, false).ctas;
  if (C % (f32 ? 4 : 8) == 0) {
    const long long v = bwd_form(C, f32, true).ctas;
    if (v > n) n = v;
  }
  if (T < n) n = T;
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
  p.w_vec = weight && al16(weight->data);
  p.b = bias ? bias->data : nullptr; p.b_f32 = bias && bias->dtype == WP_FP32;
  p.b_vec = bias && al16(bias->data);
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
  const size_t need = sums ? norm_bwd_workspace(X->rows, X->cols, X->dtype == WP_FP32) : 0;
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
  p.w_vec = weight && al16(weight->data);
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
