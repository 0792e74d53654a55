// wp_adamw.cu -- one AdamW step over the many small tensors of an adapter set.
//
//   m <- b1 m + (1 - b1) g,   v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Elementwise, so HBM is the floor; what stands between it and a set of hundreds of tensors is
// one launch per tensor.  Here a set is one launch: its table (built once, in the caller's
// memory) cuts every tensor into units of 2048 elements, a CTA takes a unit, and only the
// gradients' addresses travel with the launch, as kernel parameters.  A warp's 32 lanes hold 8
// consecutive elements each: 256 elements, one block of an 8-bit state, whose largest value is
// then one shuffle reduction.
//
// 8-bit moments: a code q of a block with scale a stands for a sign(q) (|q| / 127)^2 (m) or
// a (q / 255)^4 (v).  The power spreads the codes towards zero: the smallest m above zero is
// 6e-5 of the block's largest, the smallest v 2e-10 (its root, which divides, 1.5e-5), while the
// steps near the top stay below 1.6 %.  The codes are those of the correctly rounded float32
// sequence divide, root(s), multiply, round to even: an approximate quotient and root decide a
// code wherever they lie clear of a rounding boundary, the exact sequence where they do not.
#include <cmath>
#include <new>
#include <cstring>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

constexpr int kUnit = 2048;              // elements per CTA
constexpr int kBlock8 = 256;             // elements per 8-bit block: one warp's
constexpr int kPerLane = 8;
constexpr int kMaxGrads = WP_ADAMW_TENSORS_PER_LAUNCH;
constexpr int kInitBatch = 400;          // tensors per set-up launch

struct AdTensor {
  void* param;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  long long numel;
  int param_f32;
  int bits8;
  int vec;                               // every array allows 16-byte (8-bit codes: 8-byte) access
  int pad;
};
static_assert(sizeof(AdTensor) == 72, "layout");

struct InitParams {
  AdTensor* tensors;
  uint2* units;
  long long unit0[kInitBatch];           // first unit of each tensor, from the set's first
  int first, n;
  AdTensor t[kInitBatch];
};

struct StepParams {
  const AdTensor* tensors;
  const uint2* units;                    // (tensor, unit within it); this launch's first
  int tensor0;
  int grad_f32;
  float b1, c1, b2, c2, rb2, eps, decay, a, gs;
  const float* gs_dev;
  const void* grads[kMaxGrads];
};

__global__ void __launch_bounds__(256) adamw_init_kernel(const __grid_constant__ InitParams p) {
  const int i = blockIdx.x;
  const AdTensor& t = p.t[i];
  if (threadIdx.x == 0) p.tensors[p.first + i] = t;
  const long long n = (t.numel + kUnit - 1) / kUnit;
  for (long long u = threadIdx.x; u < n; u += blockDim.x)
    p.units[p.unit0[i] + u] = make_uint2(static_cast<uint32_t>(p.first + i), static_cast<uint32_t>(u));
}

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }

// 8 consecutive fp32 or bf16 values; n of them exist when the array has no vector access
__device__ __forceinline__ void load8(const void* p, bool f32, long long at, int n, bool vec, float (&v)[8]) {
  if (f32) {
    const float* q = static_cast<const float*>(p) + at;
    if (vec && n == 8) {
      const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? q[k] : 0.f;
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (vec && n == 8) {
      const uint4 a = *reinterpret_cast<const uint4*>(q);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = bf2f(w[k] & 0xffffu);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < n ? bf2f(q[k]) : 0.f;
    }
  }
}

__device__ __forceinline__ void store8(void* p, bool f32, long long at, int n, bool vec, const float (&v)[8]) {
  if (f32) {
    float* q = static_cast<float*>(p) + at;
    if (vec && n == 8) {
      *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = v[k];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + at;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    if (vec && n == 8) {
      st_global_v4(q, w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) q[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
    }
  }
}

__device__ __forceinline__ uint2 load_codes(const void* p, long long at, int n, bool vec) {
  const uint8_t* q = static_cast<const uint8_t*>(p) + at;
  if (vec && n == 8) return *reinterpret_cast<const uint2*>(q);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) w[k >> 2] |= static_cast<uint32_t>(q[k]) << (8 * (k & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(void* p, long long at, int n, bool vec, uint2 w) {
  uint8_t* q = static_cast<uint8_t*>(p) + at;
  if (vec && n == 8) {
    *reinterpret_cast<uint2*>(q) = w;
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) q[k] = static_cast<uint8_t>((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
}

// the codes of one word (four elements) as values; a byte becomes a float through the low
// mantissa bits of 2^23
template <bool kSigned>
__device__ __forceinline__ void decode4(uint32_t w, float top, float* v) {
  if (kSigned) w ^= 0x80808080u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + k));
    if (kSigned) {
      const float u = __fmul_rn(__fsub_rn(f, 8388608.0f + 128.0f), 1.0f / 127.0f);
      v[k] = __fmul_rn(__fmul_rn(u, fabsf(u)), top);
    } else {
      const float u = __fmul_rn(__fsub_rn(f, 8388608.0f), 1.0f / 255.0f);
      const float u2 = __fmul_rn(u, u);
      v[k] = __fmul_rn(__fmul_rn(u2, u2), top);
    }
  }
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The unrounded code of share = v / top in the root's domain, exact sequence and estimate.
template <bool kSigned>
__device__ __noinline__ float code_exact(float v, float top) {
  const float s = __fsqrt_rn(__fdiv_rn(v, top));
  return kSigned ? __fmul_rn(127.0f, s) : __fmul_rn(255.0f, __fsqrt_rn(s));
}

// Codes of this lane's 8 values in a block whose largest magnitude is top.  The estimate and the
// exact sequence each differ from the real value by the roundings of a quotient, one or two roots
// (the approximate root 2^-23) and a product: together below 4e-7 of the code, 5e-5 for m and 1e-4
// for v.  A code further than twice that from a boundary between two codes is the exact sequence's.
template <bool kSigned>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float top) {
  const bool plain = top > 1e-30f && top < 1e30f;      // the reciprocal and the estimate are normal
  const float inv = __frcp_rn(top);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float a = fabsf(v[k]);
    const float s = sqrt_approx(__fmul_rn(a, inv));
    float x = kSigned ? __fmul_rn(127.0f, s) : __fmul_rn(255.0f, sqrt_approx(s));
    const float f = x - floorf(x);
    if (!plain || fabsf(f - 0.5f) < (kSigned ? 1e-4f : 2e-4f)) {
      x = top > 0.f || top != top ? code_exact<kSigned>(a, top) : 0.f;
      if (x != x) x = 0.f;                             // such a block decodes as no finite value
    }
    if (kSigned) x = v[k] < 0.f ? -x : x;
    uint32_t q = __float_as_uint(__fadd_rn(x, 12582912.0f)) & 0xffu;   // round half to even
    if (!kSigned && q == 0 && a > 0.f) q = 1;
    w[k >> 2] |= q << (8 * (k & 3));
  }
  return make_uint2(w[0], w[1]);
}

// max that keeps a NaN (positive values compare as their bits, NaN above infinity)
__device__ __forceinline__ float warp_top(float t) {
  uint32_t u = __float_as_uint(t) & 0x7fffffffu;
  u = __reduce_max_sync(0xffffffffu, u);
  return __uint_as_float(u);
}

__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ StepParams p) {
  const uint2 unit = __ldg(p.units + blockIdx.x);
  const AdTensor t = p.tensors[unit.x];
  const void* grad = p.grads[unit.x - p.tensor0];
  if (!grad) return;
  const long long at = static_cast<long long>(unit.y) * kUnit + static_cast<long long>(threadIdx.x) * kPerLane;
  const int lane = threadIdx.x & 31;
  if (at - lane * kPerLane >= t.numel) return;         // the whole warp lies past the end
  const long long left = t.numel - at;
  const int n = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
  const bool vec = t.vec != 0;
  const bool gvec = (reinterpret_cast<uintptr_t>(grad) & 15u) == 0;

  float g[8], m[8], v[8], x[8];
  load8(grad, p.grad_f32, at, n, gvec, g);
  const bool pf32 = t.master != nullptr || t.param_f32;
  load8(t.master ? static_cast<const void*>(t.master) : t.param, pf32, at, n, vec, x);
  float* ms = nullptr;
  float* vs = nullptr;
  if (t.bits8) {
    ms = t.ms + at / kBlock8;
    vs = t.vs + at / kBlock8;
    const float mt = *ms, vt = *vs;
    const uint2 mq = load_codes(t.m, at, n, vec), vq = load_codes(t.v, at, n, vec);
    decode4<true>(mq.x, mt, m);
    decode4<true>(mq.y, mt, m + 4);
    decode4<false>(vq.x, vt, v);
    decode4<false>(vq.y, vt, v + 4);
  } else {
    load8(t.m, true, at, n, vec, m);
    load8(t.v, true, at, n, vec, v);
  }
  float gs = p.gs;
  if (p.gs_dev) gs = __fmul_rn(gs, __ldg(p.gs_dev));
  float mtop = 0.f, vtop = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float gk = __fmul_rn(g[k], gs);
    m[k] = __fadd_rn(__fmul_rn(p.b1, m[k]), __fmul_rn(p.c1, gk));
    v[k] = __fadd_rn(__fmul_rn(p.b2, v[k]), __fmul_rn(p.c2, __fmul_rn(gk, gk)));
    if (k >= n) m[k] = v[k] = 0.f;                     // elements past the end: the block's top is not theirs
    const float den = fmaf(sqrt_approx(v[k]), p.rb2, p.eps);
    x[k] = fmaf(-p.a, __fdividef(m[k], den), __fmul_rn(x[k], p.decay));
  }
  if (t.master) store8(t.master, true, at, n, vec, x);
  store8(t.param, t.param_f32, at, n, vec, x);
  if (!t.bits8) {
    store8(t.m, true, at, n, vec, m);
    store8(t.v, true, at, n, vec, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // integer maxima: a NaN stays the largest
    mtop = __uint_as_float(max(__float_as_uint(mtop), __float_as_uint(m[k]) & 0x7fffffffu));
    vtop = __uint_as_float(max(__float_as_uint(vtop), __float_as_uint(v[k]) & 0x7fffffffu));
  }
  mtop = warp_top(mtop);
  vtop = warp_top(vtop);
  store_codes(t.m, at, n, vec, encode8<true>(m, mtop));
  store_codes(t.v, at, n, vec, encode8<false>(v, vtop));
  if (lane == 0) {
    *ms = mtop;
    *vs = vtop;
  }
}

__global__ void __launch_bounds__(256) block8_decode_kernel(const uint8_t* codes, const float* absmax, long long n,
                                                            float* out, bool is_signed, bool vec) {
  const long long at = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * kPerLane;
  const long long left = n - at;
  if (left <= 0) return;
  const int cnt = left >= 8 ? 8 : static_cast<int>(left);
  const float top = __ldg(absmax + at / kBlock8);
  const uint2 w = load_codes(codes, at, cnt, vec);
  float v[8];
  if (is_signed) {
    decode4<true>(w.x, top, v);
    decode4<true>(w.y, top, v + 4);
  } else {
    decode4<false>(w.x, top, v);
    decode4<false>(w.y, top, v + 4);
  }
  store8(out, true, at, cnt, vec, v);
}

bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_tensor(const wp_adamw_tensor& t) {
  if (t.numel < 0) return WP_ERR_INVALID;
  if (t.param_dtype != WP_BF16 && t.param_dtype != WP_FP32) return WP_ERR_DTYPE;
  if (t.state_bits != 8 && t.state_bits != 32) return WP_ERR_DTYPE;
  if (t.numel == 0) return WP_OK;
  if (!t.param || !t.m || !t.v) return WP_ERR_INVALID;
  if (t.state_bits == 8 && (!t.m_absmax || !t.v_absmax)) return WP_ERR_INVALID;
  if (t.master && t.param_dtype != WP_BF16) return WP_ERR_DTYPE;
  if (!al(t.param, t.param_dtype == WP_BF16 ? 2 : 4) || !al(t.master, 4)) return WP_ERR_ALIGN;
  if (t.state_bits == 32 ? (!al(t.m, 4) || !al(t.v, 4)) : (!al(t.m_absmax, 4) || !al(t.v_absmax, 4)))
    return WP_ERR_ALIGN;
  if (t.numel > 1ll << 40) return WP_ERR_UNSUPPORTED;
  return WP_OK;
}

long long units_of(const wp_adamw_tensor& t) { return (t.numel + kUnit - 1) / kUnit; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

constexpr int kMaxTensors = WP_ADAMW_MAX_LAUNCHES * WP_ADAMW_TENSORS_PER_LAUNCH;

size_t tensors_bytes(int n) { return (static_cast<size_t>(n) * sizeof(AdTensor) + 255) & ~static_cast<size_t>(255); }

}  // namespace
}  // namespace wp

using namespace wp;

extern "C" {

size_t lora_adamw_plan_size(const wp_adamw_tensor* tensors, int32_t n) {
  if (!tensors || n < 1 || n > kMaxTensors) return 0;
  long long units = 0;
  for (int i = 0; i < n; ++i) {
    if (check_tensor(tensors[i]) != WP_OK) return 0;
    units += units_of(tensors[i]);
  }
  return tensors_bytes(n) + static_cast<size_t>(units) * sizeof(uint2) + 256;
}

int lora_adamw_plan_init(const wp_adamw_tensor* tensors, int32_t n, void* table, size_t table_bytes,
                         wp_adamw_plan* plan, void* stream) {
  if (!tensors || !plan || n < 1) return WP_ERR_INVALID;
  if (n > kMaxTensors) return WP_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i) {
    const int rc = check_tensor(tensors[i]);
    if (rc != WP_OK) return rc;
  }
  if (!table || table_bytes < lora_adamw_plan_size(tensors, n)) return WP_ERR_WORKSPACE;
  if (!al(table, 16)) return WP_ERR_ALIGN;
  wp_adamw_plan out{};
  out.table = table;
  out.n_tensors = n;
  out.n_launches = (n + kMaxGrads - 1) / kMaxGrads;
  auto* q = new (std::nothrow) InitParams;
  if (!q) return WP_ERR_INVALID;
  long long unit = 0;
  int rc = WP_OK;
  for (int first = 0; first < n && rc == WP_OK; first += kInitBatch) {
    q->tensors = static_cast<AdTensor*>(table);
    q->units = reinterpret_cast<uint2*>(static_cast<char*>(table) + tensors_bytes(n));
    q->first = first;
    q->n = n - first < kInitBatch ? n - first : kInitBatch;
    for (int i = 0; i < q->n; ++i) {
      const wp_adamw_tensor& t = tensors[first + i];
      if ((first + i) % kMaxGrads == 0) out.unit_begin[(first + i) / kMaxGrads] = unit;
      AdTensor& d = q->t[i];
      d = AdTensor{};
      d.param = t.param; d.master = t.master; d.m = t.m; d.v = t.v; d.ms = t.m_absmax; d.vs = t.v_absmax;
      d.numel = t.numel;
      d.param_f32 = t.param_dtype == WP_FP32;
      d.bits8 = t.state_bits == 8;
      const uintptr_t sa = d.bits8 ? 8 : 16;
      d.vec = al(t.param, 16) && al(t.master, 16) && al(t.m, sa) && al(t.v, sa);
      q->unit0[i] = unit;
      unit += units_of(t);
    }
    if (unit > 0x7fffffffll) {
      rc = WP_ERR_UNSUPPORTED;
      break;
    }
    adamw_init_kernel<<<q->n, 256, 0, static_cast<cudaStream_t>(stream)>>>(*q);
    rc = cuda_status(cudaGetLastError());
  }
  delete q;
  if (rc != WP_OK) return rc;
  out.unit_begin[out.n_launches] = unit;
  *plan = out;
  return WP_OK;
}

int lora_adamw_step(const wp_adamw_plan* plan, const void* const* grads, int32_t grad_dtype,
                    const wp_adamw_args* args, void* stream) {
  if (!plan || !plan->table || !grads || !args) return WP_ERR_INVALID;
  if (plan->n_tensors < 1 || plan->n_tensors > kMaxTensors ||
      plan->n_launches != (plan->n_tensors + kMaxGrads - 1) / kMaxGrads)
    return WP_ERR_INVALID;
  if (grad_dtype != WP_FP32 && grad_dtype != WP_BF16) return WP_ERR_DTYPE;
  for (double d : {args->lr, args->beta1, args->beta2, args->eps, args->weight_decay, args->grad_scale})
    if (!std::isfinite(d)) return WP_ERR_INVALID;
  if (args->beta1 < 0 || args->beta1 >= 1 || args->beta2 < 0 || args->beta2 >= 1 || args->eps < 0 || args->step < 1)
    return WP_ERR_INVALID;
  const uintptr_t ga = grad_dtype == WP_FP32 ? 4 : 2;
  for (int i = 0; i < plan->n_tensors; ++i)
    if (!al(grads[i], ga)) return WP_ERR_ALIGN;
  if (args->grad_scale_dev && !al(args->grad_scale_dev, 4)) return WP_ERR_ALIGN;
  const double t = static_cast<double>(args->step);
  StepParams p;
  p.tensors = static_cast<const AdTensor*>(plan->table);
  p.grad_f32 = grad_dtype == WP_FP32;
  p.b1 = static_cast<float>(args->beta1);
  p.c1 = static_cast<float>(1.0 - args->beta1);
  p.b2 = static_cast<float>(args->beta2);
  p.c2 = static_cast<float>(1.0 - args->beta2);
  p.rb2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(args->beta2, t)));
  p.eps = static_cast<float>(args->eps);
  p.decay = static_cast<float>(1.0 - args->lr * args->weight_decay);
  p.a = static_cast<float>(args->lr / (1.0 - std::pow(args->beta1, t)));
  p.gs = static_cast<float>(args->grad_scale);
  p.gs_dev = args->grad_scale_dev;
  const uint2* units =
      reinterpret_cast<const uint2*>(static_cast<const char*>(plan->table) + tensors_bytes(plan->n_tensors));
  for (int l = 0; l < plan->n_launches; ++l) {
    const long long u0 = plan->unit_begin[l], u1 = plan->unit_begin[l + 1];
    if (u1 <= u0) continue;
    p.tensor0 = l * kMaxGrads;
    const int n = plan->n_tensors - p.tensor0 < kMaxGrads ? plan->n_tensors - p.tensor0 : kMaxGrads;
    std::memcpy(p.grads, grads + p.tensor0, sizeof(void*) * n);
    p.units = units + u0;
    adamw_kernel<<<static_cast<unsigned>(u1 - u0), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const int rc = cuda_status(cudaGetLastError());
    if (rc != WP_OK) return rc;
  }
  return WP_OK;
}

int lora_block8_decode(const void* codes, int32_t is_signed, const float* absmax, int64_t numel, float* out,
                       void* stream) {
  if (numel < 0) return WP_ERR_INVALID;
  if (numel == 0) return WP_OK;
  if (!codes || !absmax || !out) return WP_ERR_INVALID;
  if (!al(absmax, 4) || !al(out, 4)) return WP_ERR_ALIGN;
  const long long blocks = (numel + kUnit - 1) / kUnit;
  if (blocks > 0x7fffffffll) return WP_ERR_UNSUPPORTED;
  block8_decode_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(codes), absmax, numel, out, is_signed != 0, al(codes, 8) && al(out, 16));
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
