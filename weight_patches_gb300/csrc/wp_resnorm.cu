// wp_resnorm.cu -- what stands between two blocks of a transformer, forward and backward: a block's
// output y, normed or not, gated onto the residual stream x, and the norm ahead of the next block with its
// factor and shift:
//
//   u  = (y - mu1) r1 w1  (or y),      x1 = x + alpha gate u,
//   n  = (x1 - mu2) r2,                h  = n (off + mul) + add
//
// gate, mul and add are one vector or one per sample (T / rows of the vector's matrix consecutive rows).  Backward, from
// dh and the stream's own gradient dx1, with e = dh (off + mul):
//
//   dx = dx1 + r2 (e - mean(e) - n mean(e n)),       dmul = sum dh n,  dadd = sum dh,
//   du = alpha gate dx,   dgate = sum alpha dx u,   dw1 = sum du m,  m = (y - mu1) r1,
//   dy = r1 (du w1 - mean(du w1) - m mean(du w1 m))  (or du);        no means of e and du w1 without a mean
//
// HBM bounds all of it: every row is read once and written once.  A row belongs to a CTA (to a warp where it is
// short), 8 columns to a thread, which holds them in registers as float32 pairs; it arrives by bulk copies in a ring in
// shared memory, a few rows ahead.  Forward, the CTAs' rows at a time lie together.  Backward, a worker (CTA or warp)
// takes consecutive rows, so that the sums over rows stay in its registers too: a sample that lies inside one worker's rows has
// its sums written by it; the (at most two) that reach beyond leave partial sums, which resnorm_sums_kernel adds
// in the workers' order: no atomics, the same bits each time.
//
// Measured (device time; bytes read and written once over it; a copy of as many bytes runs at 6.7 TB/s):
//   32760 x 1536, fp32 stream, bf16 block   forward 100 us, 6.0 TB/s; backward 148 us, 6.1 TB/s; with a post norm 109
//                                           and 156 (both without a mean; with means on both sides 117 and 158)
//   32760 x 1536 bf16                       forward 68 us, 5.9 TB/s; backward 107 us, 5.7 TB/s
//   16000 x 5120, fp32 stream               forward 152 us, 6.5 TB/s; backward 245 us, 6.0 TB/s
//   20000 x 4096 bf16                       forward 107 us, 6.1 TB/s; backward 166 us, 5.9 TB/s
//   100000 x 256 (a warp a row)             forward 58 us, 5.3 TB/s; backward 115 us, 4.0 TB/s
//   4000 x 16384 bf16 (two pieces a thread) forward 224 us, 2.3 TB/s; backward 354 us, 2.2 TB/s: the forms spill
//   8000 x 4099 bf16 (odd rows)             forward 83 us, 3.2 TB/s; backward 123 us, 3.2 TB/s: instructions
//   1113 x 4099 bf16, 7 samples             backward 44 us: eight rows a CTA one after another
// First forms (a row fetched a row ahead into registers): 202 and 345 us for the first line, 122 for the last.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

constexpr int kRnV = 8;                        // columns of a thread
constexpr int kRnMaxC = 16384;
constexpr int kRnWarpC = 256;                  // rows up to here belong to a warp
constexpr int kRnWarps = 8;                    // warps (rows at a time) of such a CTA
// threads up to which a CTA takes the forms of 80 (forward) and 128 (backward) registers
constexpr int kRnSmallFwd = 384, kRnSmallBwd = 512;
// and up to which the backward without a post norm takes the form of 96 (with one that spills: 205 us, 157 in the form
// of 128)
constexpr int kRnTinyBwd = 192;
// Forward, 385 to 512 threads of 8 columns: half as many of 16, so that two CTAs fit an SM and one computes at the
// other's barriers (20000 x 4096 bf16 143 -> 106 us, with a post norm 207 -> 132; up to 320 threads spill: 175).  fp32
// rows without a post norm keep the single CTA (16000 x 4096: 135.5 against 137).  Few rows take the pair, too,
// although 64 of them then need 11.4 us and not 9.3: a row's bits shall not depend on how many rows come with it.
constexpr int kRnPairFwd = 256;
// Beyond 640 threads of 8 columns: half as many of 16, in 128 registers instead of 64.  Forward 16000 x 8192 bf16 252 ->
// 160 us, fp32 stream 311 -> 242, with a post norm 330 -> 229 (not from 513 threads on: 5120 bf16 123 against 143);
// backward bf16 332 -> 283, where it spills (fp32, post norm) no gain: 524 against 525, 6144 421 against 404.
constexpr int kRnHalf = 512;
constexpr int kRnMaxStages = 4;
// What an SM has on its way from memory at a time.  More of it is worse: 32760 x 1536, fp32 stream, forward (9 KB a row)
// 2 CTAs of 3 rows 107 us, 3 of 2 99, 4 of 2 103, 4 of 4 111; backward (18 KB a row) 1 of 3 189, 2 of 2 148, 3 of 2 156,
// 3 of 4 168.
// (With a post norm a row is computed on for twice as long: half as much again, forward 121 -> 103 us.)
constexpr int kRnFlight = 70 * 1024;

// gate, mul, add, w1: row g of [rows, C], for the stream's rows g per .. (g + 1) per - 1
struct RnVec {
  const void* p;
  long long ld;
  int f32, vec;
};

struct RnParams {
  int T, C;
  int vec;                                     // 16-byte loads and stores of the rows
  const void* x; long long ldx;                // forward: x; backward: x1
  const void* y; long long ldy;
  const void* dh; long long lddh;
  const void* dx1; long long lddx1;
  void* xo; long long ldxo;                    // forward: x1; backward: dx
  void* ho; long long ldho;                    // forward: h; backward: dy
  RnVec gate, mul, add, w1;
  int gate_per, mod_per;
  float alpha, off, eps, eps1, inv_c;
  int layer, post, post_layer;
  float* stats;
  const float* stats_in;
  int workers, each, extra;
  int stages, slot;                            // the ring: rows ahead, bytes of one
  int* status;
  unsigned long long timeout_ns;
  int hold;                                    // test hook: no row is sent for, the first wait runs out
  int out_vec;                                 // 16-byte stores fit the outputs below
  float* out[4];                               // dgate, dmul, dadd, dw1
  float* part[4];                              // [workers][2][C] each
};

// 8 columns of a row as loaded: neighbours in 16-byte pieces (kVec), or every 32nd of a warp's 256, so that a
// warp's elements lie together whatever the row's address; n of them exist (all 8 but in a row's last warp)
template <typename T, bool kVec>
struct Raw8 {
  uint32_t u[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (kVec) {
      if (n == 0) return;
      const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
        const uint4 v = q[i];
        u[4 * i] = v.x; u[4 * i + 1] = v.y; u[4 * i + 2] = v.z; u[4 * i + 3] = v.w;
      }
    } else {
      using E = std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>;
      const E* q = reinterpret_cast<const E*>(p);
      uint32_t e[8];
      if (n == kRnV) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = q[i * 32];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = i < n ? q[i * 32] : 0u;
      }
#pragma unroll
      for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i)
        u[i] = sizeof(T) == 2 ? e[2 * i % 8] | (e[(2 * i + 1) % 8] << 16) : e[i];
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(2 * sizeof(T)); ++i) u[i] = 0u;
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(u[k]);
    return __uint_as_float(k & 1 ? u[k >> 1] & 0xffff0000u : u[k >> 1] << 16);
  }
  __device__ __forceinline__ F2 pair(int k) const { return f2(at(2 * k), at(2 * k + 1)); }
};

// 8 columns as float32 pairs: two operations an instruction
struct V8 {
  F2 v[kRnV / 2];
  __device__ __forceinline__ void set(float a) {
#pragma unroll
    for (int k = 0; k < kRnV / 2; ++k) v[k] = f2(a, a);
  }
  // the columns past the row's end (of a warp's strided columns) become 0
  __device__ __forceinline__ void cut(int n) {
    if (n == kRnV) return;
#pragma unroll
    for (int k = 0; k < kRnV / 2; ++k) {
      float a, b;
      f2_get(v[k], a, b);
      v[k] = f2(2 * k < n ? a : 0.f, 2 * k + 1 < n ? b : 0.f);
    }
  }
  __device__ __forceinline__ float sum() const {
    float a, b;
    f2_get(f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])), a, b);
    return a + b;
  }
  __device__ __forceinline__ void get(float (&f)[kRnV]) const {
#pragma unroll
    for (int k = 0; k < kRnV / 2; ++k) f2_get(v[k], f[2 * k], f[2 * k + 1]);
  }
};

template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* p, const V8& x, int n) {
  float v[kRnV];
  x.get(v);
  if constexpr (kVec) {
    if (n == 0) return;
    if constexpr (sizeof(T) == 2) {
      st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
    auto put = [&](int i) {
      if constexpr (sizeof(T) == 2)
        reinterpret_cast<uint16_t*>(p)[i * 32] = static_cast<uint16_t>(pack_bf16x2(v[i], 0.f));
      else
        reinterpret_cast<float*>(p)[i * 32] = v[i];
    };
    if (n == kRnV) {
#pragma unroll
      for (int i = 0; i < 8; ++i) put(i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) put(i);
    }
  }
}

// scale (off + the vector's 8 columns), or with no vector `none`
template <bool kVec>
__device__ __forceinline__ void load_vec8(const RnVec& q, long long g, int c, int n, float off, float scale, float none, V8& o) {
  if (!q.p) {
    o.set(none);
    return;
  }
  float v[kRnV];
  auto as = [&](auto raw, const auto* p) {
    raw.zero();
    raw.load(p, n);
#pragma unroll
    for (int k = 0; k < kRnV; ++k) v[k] = raw.at(k);
  };
  if (q.f32) {
    const float* p = static_cast<const float*>(q.p) + g * q.ld + c;
    if (kVec && q.vec) {
      as(Raw8<float, true>(), p);
    } else if (kVec) {
#pragma unroll
      for (int k = 0; k < kRnV; ++k) v[k] = k < n ? p[k] : 0.f;
    } else {
      as(Raw8<float, false>(), p);
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(q.p) + g * q.ld + c;
    if (kVec && q.vec) {
      as(Raw8<uint16_t, true>(), p);
    } else if (kVec) {
#pragma unroll
      for (int k = 0; k < kRnV; ++k) v[k] = k < n ? __uint_as_float(static_cast<uint32_t>(p[k]) << 16) : 0.f;
    } else {
      as(Raw8<uint16_t, false>(), p);
    }
  }
#pragma unroll
  for (int k = 0; k < kRnV / 2; ++k)
    o.v[k] = f2_mul(f2(scale, scale), f2_add(f2(off, off), f2(v[2 * k], v[2 * k + 1])));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// The rows of a CTA, on their way from memory ahead of their use: a ring of slots in shared memory, each
// the row's piece of up to four matrices one after another, filled by bulk copies that thread 0 issues.  Off the
// 16-byte path a copy takes the 16-byte pieces that hold the row, which reach into the rows before and after; the
// matrix's first and last row are loaded plainly, so that nothing outside of it is read.
struct Ring {
  uint64_t* full;
  uint8_t* slots;
  volatile int* abort_flag;
  int turn = 0;                                // the slot of the row at hand
  uint32_t phase = 0;
  __device__ __forceinline__ Ring(uint8_t* smem, int stages) {
    full = reinterpret_cast<uint64_t*>(smem);
    abort_flag = reinterpret_cast<volatile int*>(smem + kRnMaxStages * 8);
    slots = smem + kRnMaxStages * 8 + 16;
    if (stages == 0) return;
    if (threadIdx.x == 0) {
      for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
      *abort_flag = 0;
      fence_barrier_init();
    }
    __syncthreads();
  }
  // (a warp's lanes go on or leave together: shuffles follow)
  __device__ __forceinline__ bool wait(const RnParams& p) {
    return __all_sync(0xffffffffu, mbar_wait(&full[turn], phase, abort_flag, p.timeout_ns, p.status));
  }
  __device__ __forceinline__ const uint8_t* row(const RnParams& p) const { return slots + turn * p.slot; }
  __device__ __forceinline__ void next(const RnParams& p) {
    if (++turn == p.stages) {
      turn = 0;
      phase ^= 1;
    }
  }
  // thread 0: row t of matrix m to dst, as the 16-byte pieces that hold it; whether they are to be copied, or counted
  template <bool kVec, typename T>
  static __device__ __forceinline__ uint32_t piece(const void* m, long long ld, long long t, int C, uint32_t dst, uint32_t bar,
                                                   bool copy) {
    const T* at = static_cast<const T*>(m) + t * ld;
    uint32_t bytes = static_cast<uint32_t>(C) * sizeof(T);
    const char* from = reinterpret_cast<const char*>(at);
    if (!kVec) {
      const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 15u;
      from -= shift;
      bytes = (bytes + shift + 15u) & ~15u;
    }
    if (copy) bulk_load(dst, from, bytes, bar);
    return bytes;
  }
  // the row of matrix m in its place of the slot
  template <bool kVec, typename T>
  static __device__ __forceinline__ const T* at(const uint8_t* place, const void* m, long long ld, long long t) {
    if (!kVec) place += static_cast<uint32_t>(reinterpret_cast<uintptr_t>(static_cast<const T*>(m) + t * ld)) & 15u;
    return reinterpret_cast<const T*>(place);
  }
  // thread 0, after a wait ran out: the copies in flight (of `ahead` rows from the one at hand on) land before the CTA exits
  __device__ __forceinline__ void drain(const RnParams& p, int ahead) {
    for (; ahead > 0; --ahead, next(p)) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&full[turn]), phase) && globaltimer_ns() - t0 < 100000000ull) {
      }
    }
  }
};

// Sums of N (1 or 2) values over a row's threads.  red: two halves that alternate, so that one barrier a sum is
// enough.  Of two values the first shuffle leaves each half warp one.
template <int N, bool kWarp>
struct RowSum {
  float (*red)[2][32];                         // [turn][value][warp], zeros past the last warp
  int turn = 0;
  __device__ __forceinline__ explicit RowSum(float (*r)[2][32]) : red(r) {
    if constexpr (!kWarp) {
      for (int i = threadIdx.x; i < 128; i += blockDim.x) (&r[0][0][0])[i] = 0.f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x) >> 5;
    float a = v[0];
    if constexpr (N == 2) {
      const bool up = lane & 16;
      const float give = up ? v[0] : v[1];
      a = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, give, 16);
    }
#pragma unroll
    for (int o = N == 2 ? 8 : 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (kWarp) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, a, 16 * i);
      return;
    }
    if ((lane & (N == 2 ? 15 : 31)) == 0) red[turn][lane >> 4][warp] = a;
    __syncthreads();
    if (warps <= 8) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float4 p = reinterpret_cast<const float4*>(red[turn][i])[0], q = reinterpret_cast<const float4*>(red[turn][i])[1];
        v[i] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = red[turn][i][lane];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    turn ^= 1;
  }
};

// Bytes of a row's place in a slot: the row, and, off the 16-byte path, the pieces' ends.
template <typename T, bool kVec>
__host__ __device__ __forceinline__ uint32_t place_bytes(int C) {
  const uint32_t b = static_cast<uint32_t>(C) * static_cast<uint32_t>(sizeof(T));
  return kVec ? b : (b + 14u + 15u) & ~15u;
}

// The first row of worker w: rows T / workers each, the first T % workers one more.  (Rows are counted in 32
// bits: a 64-bit division costs as much as a row's sums.)
__device__ __forceinline__ int worker_begin(const RnParams& p, int w) { return p.each * w + min(w, p.extra); }
__device__ __forceinline__ int worker_of(const RnParams& p, int row) {
  const int wide = (p.each + 1) * p.extra;
  return row < wide ? row / (p.each + 1) : p.extra + (row - wide) / p.each;
}

// N: pieces of 8 columns a thread has.  kMin CTAs of kThreads fit an SM's registers.  kWarp: a row belongs to a
// warp and is loaded a row ahead; a CTA's rows travel through the ring.  kVec: 16-byte pieces fit every row.
template <typename TS, typename TY, bool kVec, bool kWarp, int N, int kThreads, int kMin>
__global__ void __launch_bounds__(kThreads, kMin) resnorm_fwd_kernel(const __grid_constant__ RnParams p) {
  constexpr bool kRing = !kWarp;
  constexpr bool kKeep = kThreads <= (N == 1 ? 640 : kRnHalf);   // a sample's vectors stay in registers
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2][2][32];
  const int lanes = kWarp ? 32 : static_cast<int>(blockDim.x);
  const int me = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int worker = kWarp ? static_cast<int>(blockIdx.x) * kRnWarps + (threadIdx.x >> 5) : static_cast<int>(blockIdx.x);
  if (worker >= p.workers) return;
  // rows worker, worker + workers, ...: the CTAs' rows at a time lie together, as DRAM's pages like them
  // (consecutive rows for each: 32760 x 1536, fp32 stream, 112.0 us; so 110.2)
  const int r0 = worker, rs = p.workers, r1 = p.T;
  constexpr int step = kVec ? 1 : 32;
  int col[N], n[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    col[j] = kVec ? (j * lanes + me) * kRnV : (j * lanes + (me & ~31)) * kRnV + (me & 31);
    n[j] = max(0, min(kRnV, (p.C - col[j] + step - 1) / step));
  }
  RowSum<1, kWarp> sum1(red);
  auto total = [&](float v) {
    float a[1] = {v};
    sum1(a);
    return a[0];
  };
  // the mean, and one over the root of the mean square about it, of v over the row; v becomes what it is
  // about its mean (and 0 in a thread past the row's end)
  auto moments = [&](V8 (&v)[N], int layer, float eps, float& mu, float& r) {
    mu = 0.f;
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) s += v[j].sum();
      mu = total(s) * p.inv_c;
      const F2 m = f2(-mu, -mu);
#pragma unroll
      for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) v[j].v[k] = f2_add(v[j].v[k], m);
        if (!kVec) v[j].cut(n[j]);
        if (kVec && n[j] == 0) v[j].set(0.f);
      }
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      F2 part = f2_mul(v[j].v[0], v[j].v[0]);
#pragma unroll
      for (int k = 1; k < kRnV / 2; ++k) part = f2_fma(v[j].v[k], v[j].v[k], part);
      float a, b;
      f2_get(part, a, b);
      q += a + b;
    }
    r = rsqrtf(fmaf(total(q), p.inv_c, eps));
  };
  constexpr int NA = kRing ? 1 : N;
  Raw8<TS, kVec> xr[N], xn[NA];
  Raw8<TY, kVec> yr[N], yn[NA];
  const uint32_t xb = place_bytes<TS, kVec>(p.C);
  auto fetch = [&](auto& x, auto& y, long long t) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      x[j].load(static_cast<const TS*>(p.x) + t * p.ldx + col[j], n[j]);
      if (p.y) y[j].load(static_cast<const TY*>(p.y) + t * p.ldy + col[j], n[j]);
    }
  };
  Ring ring(smem, kRing ? p.stages : 0);
  const bool ringed = kRing && (N == 1 || p.stages > 0);   // (the widest fp32 rows do not fit the ring)
  auto plain = [&](long long t) { return !ringed || (!kVec && (t == 0 || t == p.T - 1)); };
  auto issue = [&](long long t, int slot) {
    const uint32_t bar = smem_u32(&ring.full[slot]), dst = smem_u32(ring.slots) + slot * p.slot;
    auto all = [&](bool copy) {
      uint32_t bytes = Ring::piece<kVec, TS>(p.x, p.ldx, t, p.C, dst, bar, copy);
      if (p.y) bytes += Ring::piece<kVec, TY>(p.y, p.ldy, t, p.C, dst + xb, bar, copy);
      return bytes;
    };
    if (plain(t)) {
      mbar_arrive(&ring.full[slot]);
    } else {
      mbar_arrive_expect_tx(&ring.full[slot], all(false));
      all(true);
    }
  };
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xr[j].zero();
    yr[j].zero();
  }
  if (kRing) {
    if (threadIdx.x == 0)
      for (int i = 0; i < p.stages && r0 + i * rs < r1 && !p.hold; ++i) issue(r0 + i * rs, i);
  } else {
#pragma unroll
    for (int j = 0; j < NA; ++j) {
      xn[j].zero();
      yn[j].zero();
    }
    if constexpr (!kRing) fetch(xn, yn, r0);
  }
  if (p.w1.p)                                  // used behind the first row's sums: on its way by then
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (n[j] > 0) prefetch_l2(static_cast<const char*>(p.w1.p) + static_cast<long long>(col[j]) * (p.w1.f32 ? 4 : 2));
  V8 gate[N], mul[N], add[N];                  // alpha gate, off + mul, add
  int g = 0, m = 0, g_end = 0, m_end = 0;    // the samples that row t belongs to, their ends
  for (int t = r0; t < r1; t += rs) {
    const bool new_g = t >= g_end, new_m = t >= m_end;
    if (new_g) {
      g = t / p.gate_per;
      g_end = (g + 1) * p.gate_per;
    }
    if (new_m) {
      m = t / p.mod_per;
      m_end = (m + 1) * p.mod_per;
    }
    if (!kKeep || new_g)
#pragma unroll
      for (int j = 0; j < N; ++j) load_vec8<kVec>(p.gate, g, col[j], n[j], 0.f, p.alpha, p.alpha, gate[j]);
    if (!kKeep || new_m)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        load_vec8<kVec>(p.mul, m, col[j], n[j], p.off, 1.f, 1.f, mul[j]);
        load_vec8<kVec>(p.add, m, col[j], n[j], 0.f, 1.f, 0.f, add[j]);
      }
    if constexpr (kRing) {
      if (ringed && !ring.wait(p)) {
        if (threadIdx.x == 0) ring.drain(p, min((r1 - t + rs - 1) / rs, p.stages));
        break;
      }
      if (plain(t)) {
        fetch(xr, yr, t);
      } else {
        const uint8_t* row = ring.row(p);
        const TS* x = Ring::at<kVec, TS>(row, p.x, p.ldx, t);
        const TY* y = Ring::at<kVec, TY>(row + xb, p.y, p.ldy, t);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          xr[j].load(x + col[j], n[j]);
          if (p.y) yr[j].load(y + col[j], n[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        xr[j] = xn[j];
        yr[j] = yn[j];
      }
      if (t + rs < r1) fetch(xn, yn, t + rs);
    }
    V8 x[N];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int k = 0; k < kRnV / 2; ++k) x[j].v[k] = xr[j].pair(k);
    float mu1 = 0.f, rs1 = 0.f;
    if (p.y) {
      V8 u[N];
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) u[j].v[k] = yr[j].pair(k);
      if (p.post) {
        moments(u, p.post_layer, p.eps1, mu1, rs1);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          V8 w;
          load_vec8<kVec>(p.w1, 0, col[j], n[j], 0.f, rs1, rs1, w);
#pragma unroll
          for (int k = 0; k < kRnV / 2; ++k) u[j].v[k] = f2_mul(u[j].v[k], w.v[k]);
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) x[j].v[k] = f2_fma(gate[j].v[k], u[j].v[k], x[j].v[k]);
        if (p.xo) store8<TS, kVec>(static_cast<TS*>(p.xo) + t * p.ldxo + col[j], x[j], n[j]);
      }
    }
    float mu2, rs2;
    moments(x, p.layer, p.eps, mu2, rs2);
    if (ringed) {
      // a sum's barrier lies behind: every thread has taken the row out of its slot
      if (threadIdx.x == 0 && t + p.stages * rs < r1) issue(t + p.stages * rs, ring.turn);
      ring.next(p);
    }
    const F2 r = f2(rs2, rs2);
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int k = 0; k < kRnV / 2; ++k) x[j].v[k] = f2_fma(f2_mul(x[j].v[k], r), mul[j].v[k], add[j].v[k]);
      store8<TY, kVec>(static_cast<TY*>(p.ho) + t * p.ldho + col[j], x[j], n[j]);
    }
    if (p.stats && me == 0) {
      p.stats[t] = mu2;
      p.stats[static_cast<long long>(p.T) + t] = rs2;
      if (p.post) {
        p.stats[2ll * p.T + t] = mu1;
        p.stats[3ll * p.T + t] = rs1;
      }
    }
  }
}

// kPost: with a post norm.  A sample's vectors stay in registers where a CTA's threads leave room for them; wider rows
// read them again for each row (they lie in L1).
template <typename TS, typename TY, bool kVec, bool kWarp, bool kPost, int N, int kThreads, int kMin>
__global__ void __launch_bounds__(kThreads, kMin) resnorm_bwd_kernel(const __grid_constant__ RnParams p) {
  constexpr bool kRing = !kWarp;
  constexpr bool kKeep = N == 1 && kThreads <= 512;
  constexpr int kF = kPost ? 4 : 3;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2][2][32];
  const int lanes = kWarp ? 32 : static_cast<int>(blockDim.x);
  const int me = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int worker = kWarp ? static_cast<int>(blockIdx.x) * kRnWarps + (threadIdx.x >> 5) : static_cast<int>(blockIdx.x);
  grid_launch_dependents();                    // the sums' kernel starts as these CTAs end
  if (worker >= p.workers) return;
  const int r0 = worker_begin(p, worker), r1 = worker_begin(p, worker + 1);
  constexpr int step = kVec ? 1 : 32;
  int col[N], n[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    col[j] = kVec ? (j * lanes + me) * kRnV : (j * lanes + (me & ~31)) * kRnV + (me & 31);
    n[j] = max(0, min(kRnV, (p.C - col[j] + step - 1) / step));
  }
  RowSum<2, kWarp> sum2(red);
  V8 acc[kF][N];                               // dgate / alpha, dmul, dadd, dw1
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[f][j].set(0.f);
  // the sums of the sample that row t0 belongs to: written where all its rows are this worker's, else left
  // as the worker's first or last partial sums
  auto flush = [&](int f, V8 (&a)[N], int t0, int per, float scale) {
    if (!p.out[f]) return;
    const int g = t0 / per, begin = g * per, end = begin + per;
    const bool own = begin >= r0 && end <= r1;
    float* dst = own ? p.out[f] + static_cast<long long>(g) * p.C
                     : p.part[f] + (static_cast<long long>(worker) * 2 + (g == r0 / per ? 0 : 1)) * p.C;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float v[kRnV];
      a[j].get(v);
#pragma unroll
      for (int k = 0; k < kRnV; ++k) v[k] *= scale;
      if (kVec && (!own || p.out_vec)) {
        if (n[j] > 0) {
          reinterpret_cast<float4*>(dst + col[j])[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(dst + col[j])[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < kRnV; ++k)
          if (k < n[j]) dst[col[j] + k * step] = v[k];
      }
      a[j].set(0.f);
    }
  };
  constexpr int NA = kRing ? 1 : N;
  Raw8<TS, kVec> xr[N], sr[N], xn[NA], sn[NA];
  Raw8<TY, kVec> yr[N], hr[N], yn[NA], hn[NA];
  const uint32_t sb = place_bytes<TS, kVec>(p.C), yb = place_bytes<TY, kVec>(p.C);
  auto fetch = [&](auto& x, auto& s, auto& y, auto& h, long long t) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      h[j].load(static_cast<const TY*>(p.dh) + t * p.lddh + col[j], n[j]);
      x[j].load(static_cast<const TS*>(p.x) + t * p.ldx + col[j], n[j]);
      if (p.dx1) s[j].load(static_cast<const TS*>(p.dx1) + t * p.lddx1 + col[j], n[j]);
      if (p.y) y[j].load(static_cast<const TY*>(p.y) + t * p.ldy + col[j], n[j]);
    }
  };
  Ring ring(smem, kRing ? p.stages : 0);
  const bool ringed = kRing && (N == 1 || p.stages > 0);   // (the widest fp32 rows do not fit the ring)
  auto plain = [&](long long t) { return !ringed || (!kVec && (t == 0 || t == p.T - 1)); };
  // a slot: x1, dh, dx1, y
  auto issue = [&](long long t, int slot) {
    const uint32_t bar = smem_u32(&ring.full[slot]), dst = smem_u32(ring.slots) + slot * p.slot;
    auto all = [&](bool copy) {
      uint32_t bytes = Ring::piece<kVec, TS>(p.x, p.ldx, t, p.C, dst, bar, copy);
      bytes += Ring::piece<kVec, TY>(p.dh, p.lddh, t, p.C, dst + sb, bar, copy);
      if (p.dx1) bytes += Ring::piece<kVec, TS>(p.dx1, p.lddx1, t, p.C, dst + sb + yb, bar, copy);
      if (p.y) bytes += Ring::piece<kVec, TY>(p.y, p.ldy, t, p.C, dst + 2 * sb + yb, bar, copy);
      return bytes;
    };
    if (plain(t)) {
      mbar_arrive(&ring.full[slot]);
    } else {
      mbar_arrive_expect_tx(&ring.full[slot], all(false));
      all(true);
    }
  };
#pragma unroll
  for (int j = 0; j < N; ++j) {
    xr[j].zero();
    sr[j].zero();
    yr[j].zero();
    hr[j].zero();
  }
  if (kRing) {
    if (threadIdx.x == 0)
      for (int i = 0; i < p.stages && r0 + i < r1 && !p.hold; ++i) issue(r0 + i, i);
  }
  if constexpr (!kRing) {
#pragma unroll
    for (int j = 0; j < NA; ++j) {
      xn[j].zero();
      sn[j].zero();
      yn[j].zero();
      hn[j].zero();
    }
    fetch(xn, sn, yn, hn, r0);
  }
  V8 gate[N], mul[N], w1[kPost ? N : 1];       // alpha gate, off + mul, w1
  auto load_gate = [&](int g) {
#pragma unroll
    for (int j = 0; j < N; ++j) load_vec8<kVec>(p.gate, g, col[j], n[j], 0.f, p.alpha, p.alpha, gate[j]);
  };
  auto load_mul = [&](int m) {
#pragma unroll
    for (int j = 0; j < N; ++j) load_vec8<kVec>(p.mul, m, col[j], n[j], p.off, 1.f, 1.f, mul[j]);
  };
  auto load_w1 = [&]() {
    if constexpr (kPost)
#pragma unroll
      for (int j = 0; j < N; ++j) load_vec8<kVec>(p.w1, 0, col[j], n[j], 0.f, 1.f, 1.f, w1[j]);
  };
  if (kKeep) load_w1();
  long long g = 0, m = 0, g_end = r0, m_end = r0;   // the samples that row t belongs to, their ends
  bool failed = false;
  for (long long t = r0; t < r1; ++t) {
    if (t >= g_end) {
      if (t > r0) flush(0, acc[0], t - 1, p.gate_per, p.alpha);
      g = t / p.gate_per;
      g_end = (g + 1) * p.gate_per;
      if (kKeep) load_gate(g);
    }
    if (t >= m_end) {
      if (t > r0) {
        flush(1, acc[1], t - 1, p.mod_per, 1.f);
        flush(2, acc[2], t - 1, p.mod_per, 1.f);
      }
      m = t / p.mod_per;
      m_end = (m + 1) * p.mod_per;
      if (kKeep) load_mul(m);
    }
    if (!kKeep) load_mul(m);
    const float mu2 = p.layer ? __ldg(p.stats_in + t) : 0.f, rs2 = __ldg(p.stats_in + p.T + t);
    float mu1 = 0.f, rs1 = 0.f;
    if (kPost) {
      mu1 = p.post_layer ? __ldg(p.stats_in + 2ll * p.T + t) : 0.f;
      rs1 = __ldg(p.stats_in + 3ll * p.T + t);
    }
    if constexpr (kRing) {
      if (ringed && !ring.wait(p)) {
        if (threadIdx.x == 0) ring.drain(p, min(static_cast<int>(r1 - t), p.stages));
        failed = true;
        break;
      }
      if (plain(t)) {
        fetch(xr, sr, yr, hr, t);
      } else {
        const uint8_t* row = ring.row(p);
        const TS* x = Ring::at<kVec, TS>(row, p.x, p.ldx, t);
        const TY* h = Ring::at<kVec, TY>(row + sb, p.dh, p.lddh, t);
        const TS* s = Ring::at<kVec, TS>(row + sb + yb, p.dx1, p.lddx1, t);
        const TY* y = Ring::at<kVec, TY>(row + 2 * sb + yb, p.y, p.ldy, t);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          xr[j].load(x + col[j], n[j]);
          hr[j].load(h + col[j], n[j]);
          if (p.dx1) sr[j].load(s + col[j], n[j]);
          if (p.y) yr[j].load(y + col[j], n[j]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        xr[j] = xn[j];
        sr[j] = sn[j];
        yr[j] = yn[j];
        hr[j] = hn[j];
      }
      if (t + 1 < r1) fetch(xn, sn, yn, hn, t + 1);
    }
    // at the second norm's output: n, e = dh (off + mul)
    float s[2] = {0.f, 0.f};
    V8 x[N], d[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      // (a thread past the row's end has zeros, and keeps them)
      const float r = kVec && n[j] == 0 ? 0.f : rs2;
      F2 s0 = f2(0.f, 0.f), s1 = s0;
#pragma unroll
      for (int k = 0; k < kRnV / 2; ++k) x[j].v[k] = f2_mul(f2_add(xr[j].pair(k), f2(-mu2, -mu2)), f2(r, r));
      if (!kVec) x[j].cut(n[j]);
#pragma unroll
      for (int k = 0; k < kRnV / 2; ++k) {
        const F2 dh = hr[j].pair(k), e = f2_mul(dh, mul[j].v[k]);
        s0 = f2_fma(e, x[j].v[k], s0);
        s1 = f2_add(s1, e);
        acc[1][j].v[k] = f2_fma(dh, x[j].v[k], acc[1][j].v[k]);
        acc[2][j].v[k] = f2_add(acc[2][j].v[k], dh);
        d[j].v[k] = e;
      }
      float a, b;
      f2_get(s0, a, b);
      s[0] += a + b;
      f2_get(s1, a, b);
      s[1] += a + b;
    }
    sum2(s);
    if (ringed) {
      // the sum's barrier lies behind: every thread has taken the row out of its slot
      if (threadIdx.x == 0 && t + p.stages < r1) issue(t + p.stages, ring.turn);
      ring.next(p);
    }
    const float a1 = -s[0] * p.inv_c, a0 = p.layer ? -s[1] * p.inv_c : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float r = kVec && n[j] == 0 ? 0.f : rs2;
#pragma unroll
      for (int k = 0; k < kRnV / 2; ++k) {
        const F2 b = f2_fma(x[j].v[k], f2(a1, a1), f2_add(d[j].v[k], f2(a0, a0)));
        d[j].v[k] = p.dx1 ? f2_fma(b, f2(r, r), sr[j].pair(k)) : f2_mul(b, f2(r, r));
      }
      if (!kVec) d[j].cut(n[j]);
      if (p.xo) store8<TS, kVec>(static_cast<TS*>(p.xo) + t * p.ldxo + col[j], d[j], n[j]);
    }
    if (!p.y) continue;
    if (!kKeep) {
      load_gate(g);
      load_w1();
    }
    if constexpr (!kPost) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) {
          acc[0][j].v[k] = f2_fma(d[j].v[k], yr[j].pair(k), acc[0][j].v[k]);
          d[j].v[k] = f2_mul(d[j].v[k], gate[j].v[k]);
        }
        if (p.ho) store8<TY, kVec>(static_cast<TY*>(p.ho) + t * p.ldho + col[j], d[j], n[j]);
      }
    } else {
      // m takes n's place, e = du w1 that of dx
      float q[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float r = kVec && n[j] == 0 ? 0.f : rs1;
        F2 q0 = f2(0.f, 0.f), q1 = q0;
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) x[j].v[k] = f2_mul(f2_add(yr[j].pair(k), f2(-mu1, -mu1)), f2(r, r));
        if (!kVec) x[j].cut(n[j]);
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k) {
          const F2 m = x[j].v[k], du = f2_mul(d[j].v[k], gate[j].v[k]), e = f2_mul(du, w1[j].v[k]);
          acc[0][j].v[k] = f2_fma(f2_mul(d[j].v[k], m), w1[j].v[k], acc[0][j].v[k]);
          acc[3][j].v[k] = f2_fma(du, m, acc[3][j].v[k]);
          q0 = f2_fma(e, m, q0);
          q1 = f2_add(q1, e);
          d[j].v[k] = e;
        }
        float a, b;
        f2_get(q0, a, b);
        q[0] += a + b;
        f2_get(q1, a, b);
        q[1] += a + b;
      }
      sum2(q);
      const float b1 = -q[0] * p.inv_c, b0 = p.post_layer ? -q[1] * p.inv_c : 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int k = 0; k < kRnV / 2; ++k)
          d[j].v[k] = f2_mul(f2_fma(x[j].v[k], f2(b1, b1), f2_add(d[j].v[k], f2(b0, b0))), f2(rs1, rs1));
        if (p.ho) store8<TY, kVec>(static_cast<TY*>(p.ho) + t * p.ldho + col[j], d[j], n[j]);
      }
    }
  }
  if (failed) return;
  flush(0, acc[0], r1 - 1, p.gate_per, p.alpha);
  flush(1, acc[1], r1 - 1, p.mod_per, 1.f);
  flush(2, acc[2], r1 - 1, p.mod_per, 1.f);
  if constexpr (kPost) flush(3, acc[3], r1 - 1, p.T, 1.f);
}

// The samples that reach over several workers' rows: 32 columns and one sum (blockIdx.y) a block, a sample's
// workers shared out over its warps in order, the warps' sums added in order.  blockIdx.z counts samples, or
// (fewer) the workers in whose rows a sample begins.  32 warps where each has workers to add (one sample of 456 workers:
// 12 us with 8), 8 where samples are many, whose blocks cost more to start than they add (seven samples of 159 rows of
// 4099, 22 workers each, the backward as a whole: 58 us with 32, 46 with 8, 56 with a column a thread and no sharing).
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) resnorm_sums_kernel(const __grid_constant__ RnParams p) {
  __shared__ float red[kWarps][33];
  grid_dependency_wait();
  const int f = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!p.out[f]) return;
  const int per = f == 0 ? p.gate_per : f == 3 ? p.T : p.mod_per, groups = p.T / per;
  int g = blockIdx.z;
  if (groups <= p.workers) {
    if (g >= groups) return;
  } else {
    if (g >= p.workers) return;
    g = (worker_begin(p, g + 1) - 1) / per;     // the sample of the worker's last row
  }
  const int c0 = worker_of(p, g * per), c1 = worker_of(p, g * per + per - 1);
  if (c0 == c1 || (groups > p.workers && c0 != static_cast<int>(blockIdx.z))) return;
  const int c = blockIdx.x * 32 + lane;
  const int each = (c1 - c0 + kWarps) / kWarps;
  const int w0 = c0 + warp * each, w1 = min(c1 + 1, w0 + each);
  // the sample's first worker may have begun with another one; the others begin with it
  const int first = g == worker_begin(p, c0) / per ? 0 : 1;
  float s = 0.f;
  if (c < p.C) {
    const float* at = p.part[f] + c;
#pragma unroll 8
    for (int w = w0; w < w1; ++w) s += at[(static_cast<long long>(w) * 2 + (w == c0 ? first : 0)) * p.C];
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= p.C) return;
  s = red[0][lane];
  for (int w = 1; w < kWarps; ++w) s += red[w][lane];
  p.out[f][static_cast<long long>(g) * p.C + c] = s;
}

// ------------------------------------------------------------------ host
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// How rows of C columns are taken: a warp each, or by a CTA of `threads`, each with `pieces` times 8 columns, of
// the form of at most `form` threads; `min` of these CTAs fit an SM's registers.
struct RnShape {
  bool warp;
  int pieces, threads, form, min;
};
RnShape rn_shape(int C, bool back, bool post, bool wide) {
  if (C <= kRnWarpC) return {true, 1, 32 * kRnWarps, 32 * kRnWarps, back ? 1 : 2};
  const int pieces = C <= 8192 ? 1 : 2;
  const int threads = ((C + kRnV * pieces - 1) / (kRnV * pieces) + 31) / 32 * 32;
  const int small = back ? kRnSmallBwd : kRnSmallFwd;
  const int halves = ((C + 2 * kRnV - 1) / (2 * kRnV) + 31) / 32 * 32;
  if (pieces == 1 && threads > 640 && (!back || (!wide && !post))) return {false, 2, halves, kRnHalf, 1};
  if (pieces == 2 || threads > 640) return {false, pieces, threads, 1024, 1};
  if (!back && threads > small && threads <= 2 * kRnPairFwd && (post || !wide))
    return {false, 2, halves, kRnPairFwd, 2};
  if (threads > small) return {false, pieces, threads, 640, 1};
  if (back && !post && threads <= kRnTinyBwd) return {false, pieces, threads, kRnTinyBwd, 65536 / (threads * 112)};
  return {false, pieces, threads, small, 65536 / (threads * (back ? 128 : 80))};
}

// Workers of `min` CTAs an SM, no more than rows.
int rn_workers(long long T, const RnShape& s, int min) {
  const long long w = static_cast<long long>(std::max(1, device_sm_count())) * min * (s.warp ? kRnWarps : 1);
  return static_cast<int>(std::min<long long>(w, T));
}

// CTAs of an SM and rows of a CTA's ring, for rows of `slot` bytes: as many CTAs, two rows each at least, as keep about
// kRnFlight bytes on their way (a lone CTA up to four rows of 100 KB).
void rn_flight(const RnShape& s, int slot, bool back, bool post, int* min, int* stages) {
  const int flight = post ? kRnFlight / 2 * 3 : kRnFlight;
  *min = std::max(1, std::min(s.min, (flight + (back ? slot / 4 * 5 : 0)) / (2 * slot)));
  const int rows = *min > 1 ? (flight + 4096) / (*min * slot) : 100 * 1024 / slot;
  *stages = std::min(kRnMaxStages, std::max(2, rows));
  while (*stages > 0 && *stages * slot + 1024 > kSmemLimit) --*stages;
}

// Fills in p's workers, too.
template <typename TS, typename TY, bool kVec, bool kBack, bool kPost>
int rn_launch(RnParams& p, cudaStream_t st) {
  const RnShape s = rn_shape(p.C, kBack, p.post, sizeof(TS) == 4);
  size_t smem = 256;
  int min = s.min;
  if (!s.warp) {
    p.slot = (kBack ? 2 : 1) * static_cast<int>(place_bytes<TS, kVec>(p.C) + place_bytes<TY, kVec>(p.C));
    rn_flight(s, p.slot, kBack, p.post, &min, &p.stages);
    smem += static_cast<size_t>(p.stages) * p.slot;
  }
  p.workers = rn_workers(p.T, s, min);
  p.each = p.T / p.workers;
  p.extra = p.T % p.workers;
  const unsigned grid = s.warp ? (p.workers + kRnWarps - 1) / kRnWarps : p.workers;
  cudaError_t e = cudaSuccess;
#define WP_RN(WARP, N, TH, FMIN, BMIN)                                                                                \
  do {                                                                                                                \
    auto k = [] {                                                                                                     \
      if constexpr (kBack)                                                                                            \
        return resnorm_bwd_kernel<TS, TY, kVec, WARP, kPost, N, TH, BMIN>;                                            \
      else                                                                                                            \
        return resnorm_fwd_kernel<TS, TY, kVec, WARP, N, TH, FMIN>;                                                   \
    }();                                                                                                              \
    if (smem > 32 * 1024) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)); \
    if (e == cudaSuccess) k<<<grid, s.threads, smem, st>>>(p);                                                        \
  } while (0)
  const bool tiny = kBack && !kPost && s.form == kRnTinyBwd;
  if constexpr (kBack && !kPost)
    if (tiny) WP_RN(false, 1, kRnTinyBwd, 2, 3);
  const bool pair = !kBack && s.form == kRnPairFwd && !s.warp;
  if constexpr (!kBack)
    if (pair) WP_RN(false, 2, kRnPairFwd, 2, 1);
  constexpr bool kHalf = !kBack || (!kPost && sizeof(TS) == 2);   // as rn_shape has it
  const bool half = kHalf && s.form == kRnHalf && s.pieces == 2;
  if constexpr (kHalf)
    if (half) WP_RN(false, 2, kRnHalf, 1, 1);
  if (tiny || pair || half) {
  } else if (s.warp)
    WP_RN(true, 1, 256, 2, 1);
  else if (s.pieces == 2)
    WP_RN(false, 2, 1024, 1, 1);
  else if (s.form == 1024) {
    if constexpr (kBack && !kHalf) WP_RN(false, 1, 1024, 1, 1);   // others take two pieces a thread
  } else if (s.form == 640)
    WP_RN(false, 1, 640, 1, 1);
  else
    WP_RN(false, 1, (kBack ? kRnSmallBwd : kRnSmallFwd), 2, 1);
#undef WP_RN
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

template <typename TS, typename TY, bool kVec>
int rn_direction(RnParams& p, bool back, cudaStream_t st) {
  if (!back) return rn_launch<TS, TY, kVec, false, false>(p, st);
  return p.post ? rn_launch<TS, TY, kVec, true, true>(p, st) : rn_launch<TS, TY, kVec, true, false>(p, st);
}

int rn_dispatch(RnParams& p, bool back, bool s32, bool y32, cudaStream_t st) {
  if (s32 && y32) return p.vec ? rn_direction<float, float, true>(p, back, st) : rn_direction<float, float, false>(p, back, st);
  if (s32) return p.vec ? rn_direction<float, uint16_t, true>(p, back, st) : rn_direction<float, uint16_t, false>(p, back, st);
  return p.vec ? rn_direction<uint16_t, uint16_t, true>(p, back, st) : rn_direction<uint16_t, uint16_t, false>(p, back, st);
}

bool rows_ok(const wp_mat* m) {
  return m && m->rows >= 0 && m->cols > 0 && (m->data || m->rows == 0) && m->ld >= m->cols &&
         (m->dtype == WP_BF16 || m->dtype == WP_FP32);
}
bool rows_ok(const wp_out* m) {
  return m && m->rows >= 0 && m->cols > 0 && (m->data || m->rows == 0) && m->ld >= m->cols &&
         (m->dtype == WP_BF16 || m->dtype == WP_FP32);
}

// A vector, or one per sample
int take_vec(const wp_mat* m, long long T, long long C, RnVec* out, long long* groups) {
  if (!m) return WP_OK;
  if (!rows_ok(m) || !m->data || m->rows < 1) return WP_ERR_INVALID;
  if (m->cols != C || T % m->rows != 0) return WP_ERR_SHAPE;
  if (!aligned_element(m->data, m->dtype)) return WP_ERR_ALIGN;
  if (*groups != 0 && *groups != m->rows) return WP_ERR_SHAPE;
  *groups = m->rows;
  out->p = m->data;
  out->ld = m->ld;
  out->f32 = m->dtype == WP_FP32;
  out->vec = al16(m->data) && (m->rows == 1 || m->ld % (out->f32 ? 4 : 8) == 0);
  return WP_OK;
}

// What both directions check and set.
int rn_common(const wp_mat* X, const wp_mat* Y, const wp_residual_norm* a, RnParams* p, long long* gate_n, long long* mod_n) {
  if (!rows_ok(X) || (Y && !rows_ok(Y)) || !a) return WP_ERR_INVALID;
  if (a->kind != WP_NORM_LAYER && a->kind != WP_NORM_RMS) return WP_ERR_INVALID;
  if (a->post_kind != WP_NORM_LAYER && a->post_kind != WP_NORM_RMS && a->post_kind != WP_NORM_NONE) return WP_ERR_INVALID;
  for (double v : {a->alpha, a->mul_offset, a->eps, a->post_eps})
    if (!std::isfinite(static_cast<float>(v))) return WP_ERR_INVALID;
  if (a->eps < 0 || a->post_eps < 0) return WP_ERR_INVALID;
  if (!Y && (a->gate || a->post_weight || a->post_kind != WP_NORM_NONE)) return WP_ERR_INVALID;
  if (a->post_weight && a->post_kind == WP_NORM_NONE) return WP_ERR_INVALID;
  if (X->cols > kRnMaxC) return WP_ERR_UNSUPPORTED;
  if (Y && (Y->rows != X->rows || Y->cols != X->cols)) return WP_ERR_SHAPE;
  if (X->rows > 0x3FFFFFFFLL) return WP_ERR_UNSUPPORTED;   // rows are counted in 32 bits
  p->T = static_cast<int>(X->rows);
  p->C = static_cast<int>(X->cols);
  long long one = 0;
  *gate_n = *mod_n = 0;
  int rc;
  if ((rc = take_vec(a->gate, p->T, p->C, &p->gate, gate_n)) != WP_OK) return rc;
  if ((rc = take_vec(a->mul, p->T, p->C, &p->mul, mod_n)) != WP_OK) return rc;
  if ((rc = take_vec(a->add, p->T, p->C, &p->add, mod_n)) != WP_OK) return rc;
  if ((rc = take_vec(a->post_weight, p->T, p->C, &p->w1, &one)) != WP_OK) return rc;
  if (one > 1) return WP_ERR_SHAPE;
  p->alpha = static_cast<float>(a->alpha);
  p->off = static_cast<float>(a->mul_offset);
  p->eps = static_cast<float>(a->eps);
  p->eps1 = static_cast<float>(a->post_eps);
  p->inv_c = 1.0f / static_cast<float>(p->C);
  p->layer = a->kind == WP_NORM_LAYER;
  p->post = a->post_kind != WP_NORM_NONE;
  p->post_layer = a->post_kind == WP_NORM_LAYER;
  return WP_OK;
}

// A further matrix of the rows' sizes: its type, sizes and alignment, and whether 16-byte pieces fit it.  (The pitch decides for
// one row, too: the pieces order a row's sums, and the same row has the same bits alone and among others.)
template <typename M>
int rn_rows(const M* m, const RnParams& p, int dtype, bool* vec) {
  if (!m) return WP_OK;
  if (!rows_ok(m)) return WP_ERR_INVALID;
  if (m->dtype != dtype) return WP_ERR_DTYPE;
  if (m->rows != p.T || m->cols != p.C) return WP_ERR_SHAPE;
  if (!aligned_element(m->data, m->dtype)) return WP_ERR_ALIGN;
  *vec = *vec && al16(m->data) && m->ld % (dtype == WP_FP32 ? 4 : 8) == 0;
  return WP_OK;
}

// of the most workers that any types' rows have
size_t rn_part_bytes(long long T, int C) {
  const RnShape s = rn_shape(C, true, false, false);
  return static_cast<size_t>(rn_workers(T, s, s.min)) * 2 * C * 4;
}

}  // namespace

size_t residual_norm_bwd_workspace(long long T, long long C) {
  if (T <= 0 || C <= 0 || C > kRnMaxC) return 0;
  return 4 * rn_part_bytes(T, static_cast<int>(C));
}

}  // namespace wp

using namespace wp;

extern "C" {

int lora_residual_norm_fwd(const wp_mat* X, const wp_mat* Y, const wp_residual_norm* a, const wp_out* X_out,
                           const wp_out* H, float* stats, void* stream) {
  RnParams p{};
  long long gate_n, mod_n;
  int rc = rn_common(X, Y, a, &p, &gate_n, &mod_n);
  if (rc != WP_OK) return rc;
  if (!rows_ok(H) || (X_out && !Y)) return WP_ERR_INVALID;
  const int ydt = H->dtype;
  if (X->dtype == WP_BF16 && ydt != WP_BF16) return WP_ERR_DTYPE;
  bool vec = p.C % kRnV == 0;
  if ((rc = rn_rows(X, p, X->dtype, &vec)) != WP_OK || (rc = rn_rows(Y, p, ydt, &vec)) != WP_OK ||
      (rc = rn_rows(X_out, p, X->dtype, &vec)) != WP_OK || (rc = rn_rows(H, p, ydt, &vec)) != WP_OK)
    return rc;
  if (!aligned_element(stats, WP_FP32)) return WP_ERR_ALIGN;
  if (p.T == 0) return WP_OK;
  p.vec = vec;
  p.x = X->data; p.ldx = X->ld;
  if (Y) { p.y = Y->data; p.ldy = Y->ld; }
  if (X_out) { p.xo = X_out->data; p.ldxo = X_out->ld; }
  p.ho = H->data; p.ldho = H->ld;
  p.gate_per = static_cast<int>(p.T / std::max(1ll, gate_n));
  p.mod_per = static_cast<int>(p.T / std::max(1ll, mod_n));
  p.stats = stats;
  p.timeout_ns = device_wait_limit_ns();
  p.hold = debug_hold_flags();
  if (!(p.status = tc_status_ptr())) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  return rn_dispatch(p, false, X->dtype == WP_FP32, ydt == WP_FP32, static_cast<cudaStream_t>(stream));
}

int lora_residual_norm_bwd(const wp_mat* dH, const wp_mat* dX1, const wp_mat* X1, const wp_mat* Y, const float* stats,
                           const wp_residual_norm* a, const wp_out* dX, const wp_out* dY, const wp_out* dgate,
                           const wp_out* dmul, const wp_out* dadd, const wp_out* dpost_weight, void* workspace,
                           size_t workspace_bytes, void* stream) {
  RnParams p{};
  long long gate_n, mod_n;
  int rc = rn_common(X1, Y, a, &p, &gate_n, &mod_n);
  if (rc != WP_OK) return rc;
  if (!rows_ok(dH)) return WP_ERR_INVALID;
  if ((dgate && !a->gate) || (dmul && !a->mul) || (dpost_weight && !a->post_weight) || (dY && !Y)) return WP_ERR_INVALID;
  const int ydt = dH->dtype;
  if (X1->dtype == WP_BF16 && ydt != WP_BF16) return WP_ERR_DTYPE;
  bool vec = p.C % kRnV == 0;
  if ((rc = rn_rows(X1, p, X1->dtype, &vec)) != WP_OK || (rc = rn_rows(dH, p, ydt, &vec)) != WP_OK ||
      (rc = rn_rows(dX1, p, X1->dtype, &vec)) != WP_OK || (rc = rn_rows(Y, p, ydt, &vec)) != WP_OK ||
      (rc = rn_rows(dX, p, X1->dtype, &vec)) != WP_OK || (rc = rn_rows(dY, p, ydt, &vec)) != WP_OK)
    return rc;
  const wp_out* sums[4] = {dgate, dmul, dadd, dpost_weight};
  bool any = false;
  p.out_vec = 1;
  for (int f = 0; f < 4; ++f) {
    const wp_out* o = sums[f];
    if (!o) continue;
    if (!o->data || o->rows < 1) return WP_ERR_INVALID;
    if (o->dtype != WP_FP32) return WP_ERR_DTYPE;
    // dadd alone may say how many samples there are
    if (f == 2 && mod_n == 0) mod_n = o->rows;
    const long long rows = f == 0 ? gate_n : f == 3 ? 1 : mod_n;
    if (o->rows != rows || o->cols != p.C || p.T % rows != 0 || !one_piece(*o)) return WP_ERR_SHAPE;
    if (!aligned_element(o->data, WP_FP32)) return WP_ERR_ALIGN;
    p.out[f] = static_cast<float*>(o->data);
    p.out_vec = p.out_vec && al16(o->data);
    any = true;
  }
  if (!aligned_element(stats, WP_FP32)) return WP_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (p.T == 0) {
    for (const wp_out* o : sums) {
      if (!o) continue;
      const cudaError_t e = cudaMemsetAsync(o->data, 0, static_cast<size_t>(o->rows) * o->cols * 4, st);
      if (e != cudaSuccess) {
        set_last_cuda_error(e);
        return WP_ERR_CUDA;
      }
    }
    return WP_OK;
  }
  if (!stats) return WP_ERR_INVALID;
  if (!any && !dX && !dY) return WP_OK;
  const size_t part = rn_part_bytes(p.T, p.C);
  if (any) {
    if (!workspace || workspace_bytes < 4 * part) return WP_ERR_WORKSPACE;
    if (!al16(workspace)) return WP_ERR_ALIGN;
    for (int f = 0; f < 4; ++f) p.part[f] = reinterpret_cast<float*>(static_cast<char*>(workspace) + f * part);
  }
  p.vec = vec;
  p.x = X1->data; p.ldx = X1->ld;
  p.dh = dH->data; p.lddh = dH->ld;
  if (Y) { p.y = Y->data; p.ldy = Y->ld; }
  if (dX1) { p.dx1 = dX1->data; p.lddx1 = dX1->ld; }
  if (dX) { p.xo = dX->data; p.ldxo = dX->ld; }
  if (dY) { p.ho = dY->data; p.ldho = dY->ld; }
  p.gate_per = static_cast<int>(p.T / std::max(1ll, gate_n));
  p.mod_per = static_cast<int>(p.T / std::max(1ll, mod_n));
  p.stats_in = stats;
  p.timeout_ns = device_wait_limit_ns();
  p.hold = debug_hold_flags();
  if (!(p.status = tc_status_ptr())) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  rc = rn_dispatch(p, true, X1->dtype == WP_FP32, ydt == WP_FP32, st);
  if (rc != WP_OK || !any || p.workers == 1) return rc;
  // one group a vector, or as many blocks as samples can reach over two workers' rows
  int z = 1;
  for (int f = 0; f < 3; ++f)
    if (p.out[f]) z = std::max(z, std::min(p.T / (f == 0 ? p.gate_per : p.mod_per), p.workers));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const bool wide = p.workers / z >= 64;
  cfg.gridDim = dim3((p.C + 31) / 32, 4, static_cast<unsigned>(z));
  cfg.blockDim = dim3(wide ? 1024 : 256);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, resnorm_sums_kernel<32>, p)
                             : cudaLaunchKernelEx(&cfg, resnorm_sums_kernel<8>, p);
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

}  // extern "C"
