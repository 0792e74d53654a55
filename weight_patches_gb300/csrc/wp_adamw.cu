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
#include <algorithm>
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
  uint32_t ahead;                        // CTAs that run at a time
  int flush;                             // denormals of m and v do not reach the update
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
__device__ __forceinline__ void load8(const void* p, bool f32, long long at, int n, bool vec, F2 (&o)[4]) {
  float v[8];
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
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = f2(v[2 * k], v[2 * k + 1]);
}

__device__ __forceinline__ void store8(void* p, bool f32, long long at, int n, bool vec, const F2 (&o)[4]) {
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) f2_get(o[k], v[2 * k], v[2 * k + 1]);
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

// A sum of two products, each rounded before the sum: by the scalar add, which the compiler does not
// join with a packed product into one rounding (it did with the packed add).
__device__ __forceinline__ F2 add_each(F2 a, F2 b) {
  float ax, ay, bx, by;
  f2_get(a, ax, ay);
  f2_get(b, bx, by);
  return f2(__fadd_rn(ax, bx), __fadd_rn(ay, by));
}

// the codes of one word (four elements) as values, in pairs; a byte becomes a float through the
// low mantissa bits of 2^23
template <bool kSigned>
__device__ __forceinline__ void decode4(uint32_t w, float top, F2* v) {
  if (kSigned) w ^= 0x80808080u;
  const F2 base = kSigned ? f2(-(8388608.0f + 128.0f), -(8388608.0f + 128.0f)) : f2(-8388608.0f, -8388608.0f);
  const F2 inv = kSigned ? f2(1.0f / 127.0f, 1.0f / 127.0f) : f2(1.0f / 255.0f, 1.0f / 255.0f);
  const F2 tt = f2(top, top);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const F2 f = f2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + 2 * k)),
                    __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + 2 * k)));
    const F2 u = f2_mul(f2_add(f, base), inv);
    if (kSigned) {
      float x, y;
      f2_get(u, x, y);
      v[k] = f2_mul(f2_mul(u, f2(fabsf(x), fabsf(y))), tt);
    } else {
      const F2 u2 = f2_mul(u, u);
      v[k] = f2_mul(f2_mul(u2, u2), tt);
    }
  }
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp_approx_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// the largest, NaN when one is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The unrounded code of v / top in the root's domain, by the exact sequence.
template <bool kSigned>
__device__ __forceinline__ float code_exact(float v, float top) {
  if (!(top > 0.f || top != top)) return 0.f;
  const float s = __fsqrt_rn(__fdiv_rn(v, top));
  const float x = kSigned ? __fmul_rn(127.0f, s) : __fmul_rn(255.0f, __fsqrt_rn(s));
  return x != x ? 0.f : x;                             // such a block decodes as no finite value
}

// Codes of this lane's 8 values in a block whose largest magnitude is top.  The estimate and the
// exact sequence each differ from the real value by the roundings of a quotient, one or two roots
// (the approximate root 2^-23), each halved by every root after it, and a product.  In units of 2^-24 of the
// code, m: 1 + 2 + 1 and 0.5 + 1 + 1, together 3.9e-7, 5e-5 of a code at 127; v: 0.5 + 1 + 2 + 1 and
// 0.25 + 0.5 + 1 + 1, together 4.4e-7, 1.11e-4 at 255.  A code further than that (6e-5, 1.2e-4) from a boundary
// between two codes is the exact sequence's; the few others (one value in 8000, one in 4000) are
// formed again.
template <bool kSigned>
__device__ __forceinline__ uint2 encode8(const F2 (&v)[4], float top) {
  // inside these limits the reciprocal is normal, and a share that the estimate takes as zero for
  // being denormal has code 0 (v: 1) all the same
  const bool plain = top > 1e-24f && top < 1e30f;
  constexpr float kTop = kSigned ? 127.0f : 255.0f;
  constexpr float kSure = 0.5f - (kSigned ? 6e-5f : 1.2e-4f);
  const float i1 = __frcp_rn(top);
  const F2 inv = f2(i1, i1), magic = f2(12582912.0f, 12582912.0f), one = f2(-1.f, -1.f);
  F2 q[4];
  float worst = plain ? 0.f : 1.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float a, b;
    f2_get(f2_mul(v[k], inv), a, b);
    float x = sqrt_approx_ftz(fabsf(a)), y = sqrt_approx_ftz(fabsf(b));
    if (!kSigned) {
      x = sqrt_approx_ftz(x);
      y = sqrt_approx_ftz(y);
    }
    F2 c = f2_mul(f2(x, y), f2(kTop, kTop));
    f2_get(c, x, y);
    if (kSigned) {
      x = copysignf(x, a);
      y = copysignf(y, b);
    } else {                                           // a value above zero is never coded as zero
      f2_get(v[k], a, b);
      if (a > 0.f) x = fmaxf(x, 1.f);
      if (b > 0.f) y = fmaxf(y, 1.f);
    }
    c = f2(x, y);
    q[k] = f2_add(c, magic);                           // rounded half to even
    f2_get(f2_add(c, f2_fma(q[k], one, magic)), x, y);
    worst = fmaxf(worst, fmaxf(fabsf(x), fabsf(y)));
  }
  uint32_t w[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float x, y;
    f2_get(q[k], x, y);
    w[2 * k] = __float_as_uint(x);
    w[2 * k + 1] = __float_as_uint(y);
  }
  if (!(worst <= kSure) || !plain) {                   // a NaN among the values: plain is false
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, b;
      f2_get(v[k >> 1], a, b);
      const float z = k & 1 ? b : a, m = fabsf(z);
      float x = sqrt_approx_ftz(m * i1);
      if (!kSigned) x = sqrt_approx_ftz(x);
      x *= kTop;
      if (plain && fabsf(x - rintf(x)) <= kSure) continue;
      x = code_exact<kSigned>(m, top);
      if (!kSigned && m > 0.f) x = fmaxf(x, 1.f);
      w[k] = __float_as_uint(__fadd_rn(kSigned ? copysignf(x, z) : x, 12582912.0f));
    }
  }
  return make_uint2(__byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410));
}

// The step of this lane's n (of 8) elements from `at` on.  kFull: every lane of the warp has its 8,
// every array allows wide access and p.flush holds; all that is usual, and saves the tests and
// branches of the general form (together a third of the instructions).
template <bool kBits8, bool kFull>
__device__ __forceinline__ void step_lane(const StepParams& p, const AdTensor& t, const void* grad, long long at, int n,
                                          bool gvec) {
  const bool vec = kFull || t.vec != 0;
  if (kFull) {
    n = 8;
    gvec = true;
  }
  const bool bits8 = kBits8 && t.bits8;
  F2 g[4], m[4], v[4], x[4];
  load8(grad, p.grad_f32, at, n, gvec, g);
  load8(t.master ? static_cast<const void*>(t.master) : t.param, t.master || t.param_f32, at, n, vec, x);
  if (bits8) {
    const float mt = t.ms[at / kBlock8], vt = t.vs[at / kBlock8];
    const uint2 mq = load_codes(t.m, at, n, vec), vq = load_codes(t.v, at, n, vec);
    decode4<true>(mq.x, mt, m);
    decode4<true>(mq.y, mt, m + 2);
    decode4<false>(vq.x, vt, v);
    decode4<false>(vq.y, vt, v + 2);
  } else {
    load8(t.m, true, at, n, vec, m);
    load8(t.v, true, at, n, vec, v);
  }
  float gs = p.gs;
  if (p.gs_dev) gs = __fmul_rn(gs, __ldg(p.gs_dev));
  const F2 gs2 = f2(gs, gs), b1 = f2(p.b1, p.b1), c1 = f2(p.c1, p.c1), b2 = f2(p.b2, p.b2), c2 = f2(p.c2, p.c2);
  const F2 rb2 = f2(p.rb2, p.rb2), eps = f2(p.eps, p.eps), decay = f2(p.decay, p.decay), na = f2(-p.a, -p.a);
  float mtop = 0.f, vtop = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const F2 gk = f2_mul(g[k], gs2);
    m[k] = add_each(f2_mul(b1, m[k]), f2_mul(c1, gk));
    v[k] = add_each(f2_mul(b2, v[k]), f2_mul(c2, f2_mul(gk, gk)));
    float ma, mb, va, vb;
    f2_get(m[k], ma, mb);
    f2_get(v[k], va, vb);
    if (!kFull && n < 8) {                             // elements past the end: the block's top is not theirs
      if (2 * k >= n) ma = va = 0.f;
      if (2 * k + 1 >= n) mb = vb = 0.f;
      m[k] = f2(ma, mb);
      v[k] = f2(va, vb);
    }
    float da, db, ra, rb;
    if (kFull || p.flush) {
      f2_get(f2_fma(f2(sqrt_approx_ftz(va), sqrt_approx_ftz(vb)), rb2, eps), da, db);
      ra = ma * rcp_approx_ftz(da);
      rb = mb * rcp_approx_ftz(db);
    } else {
      f2_get(f2_fma(f2(sqrt_approx(va), sqrt_approx(vb)), rb2, eps), da, db);
      ra = __fdividef(ma, da);
      rb = __fdividef(mb, db);
    }
    x[k] = f2_fma(na, f2(ra, rb), f2_mul(x[k], decay));
    mtop = max3_nan(mtop, fabsf(ma), fabsf(mb));
    vtop = max3_nan(vtop, va, vb);
  }
  if (t.master) store8(t.master, true, at, n, vec, x);
  store8(t.param, t.param_f32, at, n, vec, x);
  if (!bits8) {
    store8(t.m, true, at, n, vec, m);
    store8(t.v, true, at, n, vec, v);
    return;
  }
  // positive values and NaN order as their bits do, NaN last
  mtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mtop) & 0x7fffffffu));
  vtop = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vtop) & 0x7fffffffu));
  store_codes(t.m, at, n, vec, encode8<true>(m, mtop));
  store_codes(t.v, at, n, vec, encode8<false>(v, vtop));
  if ((threadIdx.x & 31) == 0) {
    t.ms[at / kBlock8] = mtop;
    t.vs[at / kBlock8] = vtop;
  }
}

template <bool kBits8>
__device__ __noinline__ void step_general(const StepParams& p, uint2 unit) {
  const AdTensor t = p.tensors[unit.x];
  const void* grad = p.grads[unit.x - p.tensor0];
  const long long at = static_cast<long long>(unit.y) * kUnit + static_cast<long long>(threadIdx.x) * kPerLane;
  const long long left = t.numel - at;
  step_lane<kBits8, false>(p, t, grad, at, left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0),
                           (reinterpret_cast<uintptr_t>(grad) & 15u) == 0);
}

// Asks L2 for the unit that `p.ahead` CTAs later, about when this one ends, will be another's: its
// gradient, parameter and codes, an array a lane.
__device__ __forceinline__ void ask_ahead(const StepParams& p, uint2 unit, int lane) {
  const AdTensor& t = p.tensors[unit.x];
  const long long first = static_cast<long long>(unit.y) * kUnit;
  const long long left = t.numel - first;
  const char* base = static_cast<const char*>(lane == 2 ? t.m : t.v);
  int bytes = 1;
  if (lane == 0) {
    base = static_cast<const char*>(p.grads[unit.x - p.tensor0]);
    bytes = p.grad_f32 ? 4 : 2;
  } else if (lane == 1) {
    base = t.master ? reinterpret_cast<const char*>(t.master) : static_cast<const char*>(t.param);
    bytes = t.master || t.param_f32 ? 4 : 2;
  }
  const uint32_t size = static_cast<uint32_t>((left < kUnit ? left : kUnit) * bytes) & ~15u;
  if (base && t.bits8 && size && !(reinterpret_cast<uintptr_t>(base) & 15u))
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(base + first * bytes), "r"(size) : "memory");
}

// A unit a CTA, a block of 256 elements a warp, four CTAs' loads in flight per SM.  kBits8: whether
// the launch has 8-bit moments at all.  Measured over 57.6 million elements of 420 adapters, fp32
// gradients: 32-bit moments 237 us with fp32 parameters, 253 with bf16 ones and masters (6.8 TB/s, the copy
// rate); 8-bit 172 us with bf16 parameters and masters, 1.04 GB at 6.1 TB/s, 159 with fp32 parameters (0.92 GB,
// 5.8 TB/s).  With bf16 gradients, too, 167 us with masters (0.92 GB, 5.5 TB/s) and 149 without (0.58 GB, 3.9
// TB/s): what is left is the 8-bit step's arithmetic.  The 8-bit step is held back by its arithmetic (450 instructions per 8 elements, issue
// slots 54 % used) with the wait for loads behind it: without ask_ahead it takes 207 us; a persistent
// grid that keeps the tensor's entry between units 227 us (more registers live, fewer loads in
// flight), one that copies the next block through shared memory 238 us (its own 120 instructions).
// The 32-bit step has no use for ask_ahead.
template <bool kBits8>
__global__ void __launch_bounds__(256, 4) adamw_kernel(const __grid_constant__ StepParams p) {
  const uint2 unit = __ldg(p.units + blockIdx.x);
  uint2 ahead = unit;
  const bool ask = kBits8 && threadIdx.x < 4 && blockIdx.x + p.ahead < gridDim.x;
  if (ask) ahead = __ldg(p.units + blockIdx.x + p.ahead);
  const AdTensor t = p.tensors[unit.x];
  const void* grad = p.grads[unit.x - p.tensor0];
  if (ask) ask_ahead(p, ahead, threadIdx.x);
  if (!grad) return;
  const long long at = static_cast<long long>(unit.y) * kUnit + static_cast<long long>(threadIdx.x) * kPerLane;
  const long long first = at - (threadIdx.x & 31) * kPerLane;
  if (first >= t.numel) return;                        // the whole warp lies past the end
  const bool gvec = (reinterpret_cast<uintptr_t>(grad) & 15u) == 0;
  if (first + kBlock8 <= t.numel && t.vec && gvec && p.flush) {
    step_lane<kBits8, true>(p, t, grad, at, 8, true);
  } else {
    step_general<kBits8>(p, unit);
  }
}

// 4 consecutive codes a lane (a warp writes 512 consecutive bytes), 8 such steps a thread with their
// loads ahead.
constexpr int kDecodeSteps = 8;
__global__ void __launch_bounds__(256) block8_decode_kernel(const uint8_t* codes, const float* absmax, long long n,
                                                            float* out, bool is_signed, bool vec) {
  const long long base = static_cast<long long>(blockIdx.x) * (256 * 4 * kDecodeSteps) + threadIdx.x * 4;
  uint32_t w[kDecodeSteps];
  float top[kDecodeSteps];
#pragma unroll
  for (int k = 0; k < kDecodeSteps; ++k) {
    const long long at = base + k * 1024;
    w[k] = 0;
    top[k] = 0.f;
    if (at < n) {
      top[k] = __ldg(absmax + at / kBlock8);
      if (vec && at + 4 <= n) {
        w[k] = __ldg(reinterpret_cast<const uint32_t*>(codes + at));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (at + i < n) w[k] |= static_cast<uint32_t>(codes[at + i]) << (8 * i);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kDecodeSteps; ++k) {
    const long long at = base + k * 1024;
    if (at >= n) break;
    F2 v[2];
    if (is_signed) decode4<true>(w[k], top[k], v);
    else decode4<false>(w[k], top[k], v);
    float f[4];
    f2_get(v[0], f[0], f[1]);
    f2_get(v[1], f[2], f[3]);
    if (vec && at + 4 <= n) {
      *reinterpret_cast<float4*>(out + at) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < n) out[at + i] = f[i];
    }
  }
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

// Whether every array of the set is memory of its own: a tensor listed twice (tied parameters) would be updated
// by two CTAs at once.
int check_apart(const wp_adamw_tensor* tensors, int n) {
  struct Span {
    uintptr_t from, to;
  };
  Span* spans = new (std::nothrow) Span[static_cast<size_t>(n) * 6];
  if (!spans) return WP_ERR_INVALID;
  int count = 0;
  auto add = [&](const void* p, long long bytes) {
    if (p) spans[count++] = Span{reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(bytes)};
  };
  for (int i = 0; i < n; ++i) {
    const wp_adamw_tensor& t = tensors[i];
    if (t.numel == 0) continue;
    const long long state = t.numel * (t.state_bits == 8 ? 1 : 4);
    add(t.param, t.numel * (t.param_dtype == WP_BF16 ? 2 : 4));
    add(t.master, t.numel * 4);
    add(t.m, state);
    add(t.v, state);
    if (t.state_bits != 8) continue;
    add(t.m_absmax, (t.numel + kBlock8 - 1) / kBlock8 * 4);
    add(t.v_absmax, (t.numel + kBlock8 - 1) / kBlock8 * 4);
  }
  std::sort(spans, spans + count, [](const Span& a, const Span& b) { return a.from < b.from; });
  int rc = WP_OK;
  for (int i = 1; i < count && rc == WP_OK; ++i)
    if (spans[i].from < spans[i - 1].to) rc = WP_ERR_INVALID;
  delete[] spans;
  return rc;
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
  const int apart = check_apart(tensors, n);
  if (apart != WP_OK) return apart;
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
      if (t.state_bits == 8) out.launches_8bit |= 1u << ((first + i) / kMaxGrads);
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
  p.ahead = 4u * device_sm_count();
  p.b1 = static_cast<float>(args->beta1);
  p.c1 = static_cast<float>(1.0 - args->beta1);
  p.b2 = static_cast<float>(args->beta2);
  p.c2 = static_cast<float>(1.0 - args->beta2);
  p.rb2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(args->beta2, t)));
  p.eps = static_cast<float>(args->eps);
  p.decay = static_cast<float>(1.0 - args->lr * args->weight_decay);
  // sqrt(v) of a denormal v is below 1.1e-19: here rb2 times that is less than half a unit in eps's
  // last place, and a denormal m moves the parameter by less than 4e-27 of the rate.  So the roots
  // and quotients that take denormals as zero, without the scaling around the others, are used.
  p.flush = p.rb2 * 3.7e-12f <= p.eps;
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
    const unsigned n_units = static_cast<unsigned>(u1 - u0);
    if (plan->launches_8bit >> l & 1u) adamw_kernel<true><<<n_units, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
    else adamw_kernel<false><<<n_units, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
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
  const long long blocks = (numel + 1024 * kDecodeSteps - 1) / (1024 * kDecodeSteps);
  if (blocks > 0x7fffffffll) return WP_ERR_UNSUPPORTED;
  block8_decode_kernel<<<static_cast<unsigned>(blocks), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(codes), absmax, numel, out, is_signed != 0, al(codes, 4) && al(out, 16));
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
