// wp_norm.cu -- layer norm and the form without a mean, forward and backward.
//
//   forward   y = (x - mu) r w + b,  r = 1 / sqrt(var + eps)
//   backward  xh = (x - mu) r, h = dy w
//             dx = r (h - mean(h) - xh mean(h xh))       (no mean(h) without a mean)
//             dw = sum_t dy xh,  db = sum_t dy
//
// Both are bound by HBM.  Rows travel by bulk copies into a ring of row slots in shared memory,
// several rows ahead, so that the bytes in flight do not depend on how many registers the
// arithmetic takes; a row is then held in registers, its sums are taken there (the squares after
// the mean is out, so that a large mean costs no digits), and it is written once.  The arithmetic runs
// on float32 pairs (two operations per instruction).  Rows of any length and alignment travel the
// same way: the copy takes the 16-byte pieces that hold them, each thread picks its vector of columns
// out of two pieces, and on the way out shuffles bring the vectors back to 16-byte pieces.
// Forward: a CTA works through its rows, one warp where a row is short.  Backward: a CTA's threads
// keep their columns over all of its rows, so the column sums dw and db stay in registers; each
// CTA leaves one partial row of them in the workspace, which a second kernel adds in order: no
// atomics, the same bits each time.
//
// Measured (device time; bytes read and written once over it; a copy reaches 6.8 TB/s):
//   32760 x 1536 bf16   forward 34 us, 5.9 TB/s; backward 57 us, 5.3 TB/s, the first rows' arrival and the
//                       second kernel included
//   16000 x 5120 fp32   forward 114 us, 5.8 TB/s; backward 153 us, 6.4 TB/s
//   16 x 5120 bf16      forward 3.5 us, of which a launch is most
//   20000 x 2187 bf16   forward 70 us, 2.5 TB/s; backward 116 us, 2.3 TB/s: the shifts, twice the
//                       arithmetic of an aligned row, are what bounds these
//   8000 x 4099 fp32    forward 93 us, 2.8 TB/s; backward 124 us, 3.2 TB/s
// Shifted rows were read and written element by element first: 96 and 278 us, 102 and 161 us.  Their
// backward takes half the rows a turn of an aligned one's: with as many, the registers spill.
// The widest forms spill all the same (bytes a thread): the backward's of 32 elements 144 to 664 bf16, 192 to
// 592 fp32, its shifted one of 24 120 to 288, the bf16 forward's of 32 72 to 208; others up to 48.
//   8192 x 12288 bf16   forward 83 us, 4.8 TB/s; backward 137 us, 4.4 TB/s (24 elements a thread)
//   8192 x 14336 bf16   forward 93 us, 5.0 TB/s; backward 203 us, 3.5 TB/s
//   8192 x 12288 fp32   forward 277 us, 2.9 TB/s; backward 299 us, 4.0 TB/s
// Rows beyond the registers of 512 threads (32768 columns of bf16 forward, 16384 of any other) or of which the
// ring does not hold two turns (fp32 backward, from 13953 columns on) are read once per sum, element by
// element: 2000 x 40000 bf16 forward 284 us, backward 961; fp32 392 and 1002, 8192 x 14336 fp32 backward 1032.
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
  int stages, slot;                // the CTA's ring of rows: stages, bytes of a row's slot
  int* status;
  unsigned long long timeout_ns;
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

// Sums of N values (a power of two) over the CTA; red holds N per warp and is not used by the sum
// before (the callers alternate two).  A CTA barrier; `fail` becomes whether any thread passed it
// true.  Within a warp the lanes share the values out as they add (each step halves what a lane
// still carries), so N values cost N - 1 shuffles and the steps left, not 5 N; across the warps each
// group of N lanes adds its share of the warps' sums, and the groups meet by shuffles.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float* red, bool& fail) {
  constexpr int kLog = N == 1 ? 0 : N == 2 ? 1 : N == 4 ? 2 : 3;
  static_assert(N == 1 << kLog, "1, 2, 4 or 8 values");
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int b = 0; b < kLog; ++b) {
    const int o = 16 >> b, half = N >> (b + 1);
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int o = 16 >> kLog; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  // lane l holds value l >> (5 - kLog) of its warp
  if (warps == 1) {
    fail = __any_sync(0xffffffffu, fail);
    const float t = v[0];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i << (5 - kLog));
    return;
  }
  if ((lane & ((32 >> kLog) - 1)) == 0) red[(threadIdx.x >> 5) * N + (lane >> (5 - kLog))] = v[0];
  fail = __syncthreads_or(fail);
  float t = 0.f;
  for (int w = lane >> kLog; w < warps; w += 32 >> kLog) t += red[w * N + (lane & (N - 1))];
#pragma unroll
  for (int o = 16; o >= N; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = N == 1 ? t : __shfl_sync(0xffffffffu, t, i);
}

constexpr int kMaxThreads = 512;
constexpr int kMaxStages = 8;
constexpr int kSmemPerSm = 220 * 1024;

// A thread's columns come in chunks of one vector of V elements; their values are pairs.
template <int V>
struct Chunk {
  static constexpr int kPairs = V / 2;
  F2 p[kPairs];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) p[k] = f2(0.f, 0.f);
  }
  // the elements past the first n
  __device__ __forceinline__ void cut(int n) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      float a, b;
      f2_get(p[k], a, b);
      p[k] = f2(2 * k < n ? a : 0.f, 2 * k + 1 < n ? b : 0.f);
    }
  }
};

// How the rows lie.  kExact: 16-byte aligned, and every thread has all of its chunks.  kWhole: aligned,
// of whole vectors.  kShifted: any alignment and length.  There a warp's chunks are neighbours, so that
// shuffles can bring a row's vectors to the 16-byte pieces that they are stored in.
enum { kExact = 0, kWhole = 1, kShifted = 2 };

// first column of chunk i of NC
template <int V, int NC, int kMode>
__device__ __forceinline__ int chunk_col(int i) {
  if (kMode == kShifted)
    return ((static_cast<int>(threadIdx.x >> 5) * NC + i) * 32 + static_cast<int>(threadIdx.x & 31)) * V;
  return (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * V;
}

// The 16 bytes from byte `sh` (0 to 15, the same in a warp) of the first six of eight words, those
// words taken from the eight by bit 3 already.
template <typename T>
__device__ __forceinline__ void window(const uint32_t (&b)[6], uint32_t sh, uint32_t (&o)[4]) {
  uint32_t c[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) c[k] = sh & 4 ? b[k + 1] : b[k];
  if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = c[k];
  } else {
    const uint32_t sel = sh & 2 ? 0x5432u : 0x3210u;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __byte_perm(c[k], c[k + 1], sel);
  }
}

__device__ __forceinline__ float f2_sum(F2 a) {
  float x, y;
  f2_get(a, x, y);
  return x + y;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// What of rows r to r + n - 1, which lie one after another (or n is 1), travels by bulk copy: the 16-byte
// pieces that hold them, into shared memory at the same offset from a 16-byte boundary.  The outermost
// pieces reach into the rows before and after, so the matrix's first row leaves out its first piece
// where that is not all its own, and the last row its last: those elements are patched in.  (At first
// every row's ends were read from global memory: the wait for them, once a turn, took most of the time.)
template <typename T>
struct RowSpan {
  const T* row;
  int lo, hi;                            // elements [lo, hi) of the n C travel
  uintptr_t from;                        // the copy's source and bytes
  uint32_t skip;                         // bytes from the row's 16-byte boundary to the copy's start
  uint32_t bytes;
  __device__ __forceinline__ RowSpan(const T* base, long long ld, long long r, int n, long long rows, int C)
      : row(base + r * ld) {
    const int len = n * C;
    const uintptr_t b = reinterpret_cast<uintptr_t>(row), e = b + static_cast<uintptr_t>(len) * sizeof(T);
    lo = 0;
    hi = len;
    skip = 0;
    const bool tiny = ld * static_cast<long long>(sizeof(T)) < 16;
    from = b & ~static_cast<uintptr_t>(15);
    uintptr_t to = (e + 15) & ~static_cast<uintptr_t>(15);
    if ((b & 15u) && (r == 0 || tiny)) {
      from += 16;
      skip = 16;
    }
    if (r + n == rows || tiny) to = e & ~static_cast<uintptr_t>(15);
    bytes = to > from ? static_cast<uint32_t>(to - from) : 0;
    if (!bytes) {
      lo = hi = len;
    } else {
      if (from > b) lo = static_cast<int>((from - b) / sizeof(T));
      if (to < e) hi = static_cast<int>((to - b) / sizeof(T));
    }
  }
};

// The CTA's walk: turn after turn of ROWS rows, through a ring of stages that each hold those rows
// of OPS matrices.  A stage is filled with bulk copies: one for the turn's rows of a matrix where they
// lie one after another (they do in shared memory then, too), else one a row, into slots; kShifted
// works its spans out a lane each (one thread took a microsecond a turn for them).  A stage may be
// filled again once every thread has read it (the callers pass a CTA barrier in between).  Row numbers
// are 32-bit, offsets 64-bit; pointers step from turn to turn.
template <typename T, int kMode, int ROWS, int OPS>
struct Walk {
  const NormParams& p;
  uint64_t* full;
  uint32_t base;                         // shared-memory address of this turn's stage
  int s;
  uint32_t phase;
  int row, step;                         // this turn's first row; rows between turns

  __device__ __forceinline__ Walk(const NormParams& p_, void* mem, uint64_t* full_)
      : p(p_), full(full_), base(smem_u32(mem)), s(0), phase(0), row(static_cast<int>(blockIdx.x) * ROWS),
        step(static_cast<int>(gridDim.x) * ROWS) {}
  __device__ __forceinline__ int total() const { return static_cast<int>(p.T); }
  __device__ __forceinline__ uint32_t stage_bytes() const { return static_cast<uint32_t>(p.slot) * (ROWS * OPS); }
  __device__ __forceinline__ bool more() const { return row < total(); }
  __device__ __forceinline__ bool joined() const { return p.ldx == p.C && (OPS == 1 || p.lddy == p.C); }
  __device__ __forceinline__ void next() {
    row = total() - row > step ? row + step : total();
    base += stage_bytes();
    if (++s == p.stages) {
      s = 0;
      phase ^= 1;
      base -= static_cast<uint32_t>(p.stages) * stage_bytes();
    }
  }
  // shared-memory address of slot j of operand o in this turn's stage
  __device__ __forceinline__ uint32_t at(int j, int o) const {
    return base + static_cast<uint32_t>((o * ROWS + j) * p.slot);
  }
  __device__ __forceinline__ RowSpan<T> span(int o, long long r, int n) const {
    return RowSpan<T>(static_cast<const T*>(o == 0 ? p.x : p.dy), o == 0 ? p.ldx : p.lddy, r, n, p.T, p.C);
  }
  __device__ __forceinline__ const T* src(int o, long long r) const {
    return o == 0 ? static_cast<const T*>(p.x) + r * p.ldx : static_cast<const T*>(p.dy) + r * p.lddy;
  }
  // the rows from r0 (64-bit: it may lie past the end) into the stage at `dst` (warp 0)
  __device__ __forceinline__ void fill(uint32_t dst, int stage, long long r0) const {
    if (r0 >= p.T) return;
    const int n = p.T - r0 < ROWS ? static_cast<int>(p.T - r0) : ROWS;
    if constexpr (kMode != kShifted) {
      if (threadIdx.x != 0) return;
      mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(n * OPS * p.C) * sizeof(T));
      for (int o = 0; o < OPS; ++o) {
        const uint32_t d = dst + static_cast<uint32_t>(o * ROWS * p.slot);
        if ((o == 0 ? p.ldx : p.lddy) == p.C) {
          bulk_load(d, src(o, r0), static_cast<uint32_t>(n * p.C) * sizeof(T), &full[stage]);
          continue;
        }
        for (int j = 0; j < n; ++j)
          bulk_load(d + j * p.slot, src(o, r0 + j), static_cast<uint32_t>(p.C) * sizeof(T), &full[stage]);
      }
      return;
    }
    const int lane = threadIdx.x & 31;
    const bool one = joined();
    const int o = one ? lane : lane / ROWS, j = one ? 0 : lane % ROWS;
    uint64_t* bar = &full[stage];
    const bool mine = o < OPS && j < n;
    const RowSpan<T> q = span(mine ? o : 0, r0 + (mine ? j : 0), one ? n : 1);
    const uint32_t bytes = mine ? q.bytes : 0;
    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
    if (lane == 0) mbar_arrive_expect_tx(bar, all);
    __syncwarp();
    if (bytes)
      bulk_load(dst + static_cast<uint32_t>((o * ROWS + j) * p.slot) + q.skip, reinterpret_cast<const void*>(q.from), bytes,
                bar);
  }
  __device__ __forceinline__ void refill() const {       // this turn's stage, `stages` turns on
    if (threadIdx.x < (kMode == kShifted ? 32 : 1)) fill(base, s, row + static_cast<long long>(step) * p.stages);
  }
  // Barriers, then the first `stages` turns on their way.
  __device__ __forceinline__ void begin(volatile int* abort_flag) const {
    if (threadIdx.x < 32) {
      if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
      }
      __syncwarp();
      for (int i = 0; i < p.stages; ++i) fill(base + i * stage_bytes(), i, row + static_cast<long long>(step) * i);
    }
    __syncthreads();
  }
  // Shared-memory address of column 0 of row j of operand o (a row past the end: its slot's start, which
  // lies behind the rows there are).
  __device__ __forceinline__ uint32_t column0(int j, int o) const {
    if (row + j >= total()) return at(j, o);
    if (kMode != kShifted) return at(j, o);
    const uint32_t pitch = static_cast<uint32_t>(p.C) * static_cast<uint32_t>(sizeof(T));
    const bool one = joined();
    const uint32_t a = one ? at(0, o) + static_cast<uint32_t>(j) * pitch : at(j, o);
    const uint32_t b = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(o == 0 ? p.x : p.dy));
    const uint32_t ld = static_cast<uint32_t>(o == 0 ? p.ldx : p.lddy);
    return a + ((b + static_cast<uint32_t>(one ? row : row + j) * ld * static_cast<uint32_t>(sizeof(T))) & 15u);
  }
  // What the copies left out of the first and last rows, by plain loads (a CTA barrier in their turns
  // only).
  __device__ __forceinline__ void patch() const {
    if (kMode != kShifted) return;
    const bool tiny = (OPS == 2 && p.lddy < p.ldx ? p.lddy : p.ldx) * static_cast<long long>(sizeof(T)) < 16;
    const int n = total() - row < ROWS ? total() - row : ROWS;
    if (row != 0 && row + n != total() && !tiny) return;
    const bool one = joined();
    for (int o = 0; o < OPS; ++o)
      for (int j = 0; j < (one ? 1 : n); ++j) {
        const RowSpan<T> q = span(o, row + j, one ? n : 1);
        const int len = one ? n * p.C : p.C;
        for (int i = threadIdx.x; i < q.lo + len - q.hi; i += blockDim.x) {
          const int c = i < q.lo ? i : q.hi + i - q.lo;
          if (c >= len) break;
          const uint32_t to = column0(j, o) + static_cast<uint32_t>(c) * static_cast<uint32_t>(sizeof(T));
          if (sizeof(T) == 2)
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(reinterpret_cast<const uint16_t*>(q.row)[c]) : "memory");
          else
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(reinterpret_cast<const uint32_t*>(q.row)[c]) : "memory");
        }
      }
    fence_proxy_async_smem();            // the stage is filled by a copy again
    __syncthreads();
  }
  // The last turn may hold fewer than ROWS rows: the missing ones read as zeros, so that the turn
  // needs no tests (a CTA barrier in that turn only).
  __device__ __forceinline__ void pad() const {
    patch();
    const int n = total() - row;
    if (n >= ROWS) return;
    for (int o = 0; o < OPS; ++o)
      for (uint32_t b = threadIdx.x * 4; b < static_cast<uint32_t>((ROWS - n) * p.slot); b += blockDim.x * 4)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at(n, o) + b), "r"(0) : "memory");
    __syncthreads();
  }
  // After an expired wait: the copies still in flight land before the CTA leaves (this turn's and
  // those of the stages - 1 turns after it).
  __device__ __forceinline__ void settle() {
    if (threadIdx.x != 0) return;
    for (int k = 0; k < p.stages && more(); ++k, next()) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&full[s]), phase) && globaltimer_ns() - t0 < 100000000ull) {
      }
    }
  }
};

// Chunk i of a row as loaded, and its values.
template <typename T, int V>
struct RawChunk {
  uint32_t u[4];
  // from column c, at shared-memory address `at`; n columns exist from there on
  template <int kMode>
  __device__ __forceinline__ void load(uint32_t at, int n) {
    if constexpr (kMode != kShifted) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                   : "r"(at));
    } else {
      uint32_t b[6];
#pragma unroll
      for (int k = 0; k < 3; ++k)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(b[2 * k]), "=r"(b[2 * k + 1]) : "r"((at & ~7u) + 8 * k));
      window<T>(b, at, u);
      if (n < V) {
        asm volatile("" ::: "memory");     // a branch that few warps take, not selects in all
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (sizeof(T) == 4) u[k] = k < n ? u[k] : 0u;
          else u[k] = 2 * k + 1 < n ? u[k] : 2 * k < n ? u[k] & 0xffffu : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ Chunk<V> values() const {
    Chunk<V> o;
#pragma unroll
    for (int k = 0; k < Chunk<V>::kPairs; ++k) {
      if constexpr (V == 8) o.p[k] = f2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
      else o.p[k] = f2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1]));
    }
    return o;
  }
};

// The chunk at column c of a weight or bias vector (zero where there is no column)
template <int V>
__device__ __forceinline__ Chunk<V> vec_chunk(const void* p, int f32, int vec, int c, int C) {
  Chunk<V> o;
  float t[V];
  if (c + V <= C) {
    load_vec<V>(p, f32, vec, c, t);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float q[1] = {0.f};
      if (c + k < C) load_vec<1>(p, f32, 0, c + k, q);
      t[k] = q[0];
    }
  }
#pragma unroll
  for (int k = 0; k < V / 2; ++k) o.p[k] = f2(t[2 * k], t[2 * k + 1]);
  return o;
}

template <typename T, int V>
__device__ __forceinline__ void store_chunk(T* row, const Chunk<V>& x, int c) {
  float o[V];
#pragma unroll
  for (int k = 0; k < V / 2; ++k) f2_get(x.p[k], o[2 * k], o[2 * k + 1]);
  store_row<T, V>(row + c, o);
}

// A row of any alignment, stored by a warp chunk after chunk (all lanes call for every chunk).  The row's
// 16-byte piece at a vector's column holds the last s elements of the vector before it and the first
// V - s of its own: the lane before gives its words (the last lane those of the chunk before).  At a
// warp's two ends a piece is another warp's in part: each stores its part in 2, 4 and 8 bytes.  The
// row's last piece goes element by element.
template <typename T, int V, int NC, int kMode>
struct ShiftedStore {
  T* row;
  uint32_t off;                          // bytes from a 16-byte boundary to column 0, and to any vector
  int s;
  uint32_t last[4];                      // the chunk before, of lane 31 (lane 0's neighbour)
  __device__ __forceinline__ explicit ShiftedStore(T* r)
      : row(r), off(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r)) & 15u),
        s(static_cast<int>(off) / static_cast<int>(sizeof(T))) {}
  __device__ __forceinline__ void shift(const uint32_t (&a)[8], uint32_t (&o)[4]) const {
    const uint32_t sh = 16u - off;
    uint32_t b[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) b[k] = sh & 8 ? a[k + 2] : a[k];
    window<T>(b, sh, o);
  }
  __device__ __forceinline__ void put(const Chunk<V>& x, int i, int C, bool live) {
    const int lane = threadIdx.x & 31, c = chunk_col<V, NC, kMode>(i);
    uint32_t a[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x0, x1;
      if constexpr (V == 8) {
        f2_get(x.p[k], x0, x1);
        a[4 + k] = pack_bf16x2(x0, x1);
      } else {
        f2_get(x.p[k >> 1], x0, x1);
        a[4 + k] = __float_as_uint(k & 1 ? x1 : x0);
      }
    }
    char* piece = reinterpret_cast<char*>(row + c) - off;
    if (off == 0) {
      if (live && c + V <= C) st_global_v4(piece, a[4], a[5], a[6], a[7]);
      if (live && c + V > C) put_elements(a, c, 0, C - c);
      return;
    }
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t give = lane == 31 && i > 0 ? last[k] : a[4 + k];
      a[k] = __shfl_sync(0xffffffffu, give, (lane + 31) & 31);
      last[k] = a[4 + k];
    }
    shift(a, o);
    const int left = C - (c - s);        // elements from the piece's first on
    if (!live) return;
    if ((lane > 0 || i > 0) && left >= V) st_global_v4(piece, o[0], o[1], o[2], o[3]);
    if (i == 0 && lane == 0 && left >= V) {        // bytes [off, 16) of the piece
      asm volatile("" ::: "memory");
      if (sizeof(T) == 2 && (off & 2)) *reinterpret_cast<uint16_t*>(piece + off) = static_cast<uint16_t>(pick(o, off >> 2) >> 16);
      const uint32_t w = (off + 3) >> 2;
      if (w & 1) *reinterpret_cast<uint32_t*>(piece + 4 * w) = w == 1 ? o[1] : o[3];
      if (w <= 2) *reinterpret_cast<uint2*>(piece + 8) = make_uint2(o[2], o[3]);
    }
    if (i == NC - 1 && lane == 31 && c + V <= C) { // bytes [0, off) of the next piece
      asm volatile("" ::: "memory");
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = a[4 + k];
      shift(a, o);
      piece += 16;
      if (off & 8) *reinterpret_cast<uint2*>(piece) = make_uint2(o[0], o[1]);
      if (off & 4) *reinterpret_cast<uint32_t*>(piece + (off & 8)) = off & 8 ? o[2] : o[0];
      if (sizeof(T) == 2 && (off & 2)) *reinterpret_cast<uint16_t*>(piece + (off & 12)) = static_cast<uint16_t>(pick(o, off >> 2));
      return;
    }
    // the row's last vector: its elements in a piece that no vector store covers
    const bool next = (lane < 31 || i < NC - 1) && left >= 2 * V;
    if (left < V || !next) {
      asm volatile("" ::: "memory");
      put_elements(a, c, left < V ? 0 : V - s, C - c);
    }
  }
  __device__ __forceinline__ static uint32_t pick(const uint32_t (&o)[4], uint32_t w) {
    const uint32_t lo = w & 1 ? o[1] : o[0], hi = w & 1 ? o[3] : o[2];
    return w & 2 ? hi : lo;
  }
  // own elements k with from <= k < n
  __device__ __forceinline__ void put_elements(const uint32_t (&a)[8], int c, int from, int n) const {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (k < from || k >= n) continue;
      if constexpr (V == 8) reinterpret_cast<uint16_t*>(row + c)[k] = static_cast<uint16_t>(a[4 + (k >> 1)] >> (16 * (k & 1)));
      else reinterpret_cast<uint32_t*>(row + c)[k] = a[4 + k];
    }
  }
};

// A chunk of the partial column sums (rows of C floats, of any alignment)
template <int V>
__device__ __forceinline__ void store_sums(float* row, const Chunk<V>& x, int c, int C) {
#pragma unroll
  for (int k = 0; k < Chunk<V>::kPairs; ++k) {
    float a, b;
    f2_get(x.p[k], a, b);
    if (c + 2 * k < C) row[c + 2 * k] = a;
    if (c + 2 * k + 1 < C) row[c + 2 * k + 1] = b;
  }
}

// The chunks of a weight or bias vector that a thread's columns need: kept in registers for all rows
// as values (kHeldValues) or, for bf16 vectors that would not fit beside the rows as values, packed
// as loaded (kHeldPacked, V = 8); or loaded again at each use (kHeldNot), which exposes a load's
// latency every turn.
enum { kHeldNot = 0, kHeldValues = 1, kHeldPacked = 2 };
template <int V, int NC, int kHeld, int kMode>
struct Held {
  Chunk<V> c[kHeld == kHeldValues ? NC : 1];
  RawChunk<uint16_t, V> r[kHeld == kHeldPacked ? NC : 1];
  const void* p;
  int f32, vec, C;
  float none;                            // what a missing vector stands for (1 or 0)
  __device__ __forceinline__ Held(const void* p_, int f32_, int vec_, int C_, float none_)
      : p(p_), f32(f32_), vec(vec_), C(C_), none(none_) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (kHeld == kHeldValues) c[kHeld == kHeldValues ? i : 0] = load(i);
      if constexpr (kHeld == kHeldPacked && V == 8) {
        const uint32_t w = none != 0.f ? 0x3f803f80u : 0u;
        uint4 q = make_uint4(w, w, w, w);
        const int at = chunk_col<V, NC, kMode>(i);
        if (p && at + V <= C) {
          q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
        } else if (kMode == kShifted && p) {
          uint32_t h[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) h[k] = at + k < C ? __ldg(static_cast<const unsigned short*>(p) + at + k) : 0u;
          q = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
        r[i].u[0] = q.x; r[i].u[1] = q.y; r[i].u[2] = q.z; r[i].u[3] = q.w;
      }
    }
  }
  __device__ __forceinline__ Chunk<V> load(int i) const {
    Chunk<V> o;
    const int at = chunk_col<V, NC, kMode>(i);
    if (p && at < C) return vec_chunk<V>(p, f32, vec, at, C);
#pragma unroll
    for (int k = 0; k < Chunk<V>::kPairs; ++k) o.p[k] = f2(none, none);
    return o;
  }
  __device__ __forceinline__ Chunk<V> at(int i) const {
    if constexpr (kHeld == kHeldPacked) return r[i].values();
    else return kHeld == kHeldValues ? c[kHeld == kHeldValues ? i : 0] : load(i);
  }
};

// Forward, ROWS rows of a CTA per turn (a CTA is one warp where that is enough); NC chunks a thread.
template <typename T, int V, int NC, int ROWS, int kHeld, int kRegs, int kMode>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__(kRegs) norm_fwd_kernel(const NormParams p, const bool layer) {
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[2][16 * ROWS];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_word;
  constexpr int P = Chunk<V>::kPairs;
  Walk<T, kMode, ROWS, 1> walk(p, ring_mem, full);
  walk.begin(&abort_word);
  const Held<V, NC, kHeld, kMode> w(p.w, p.w_f32, p.w_vec, p.C, 1.f), b(p.b, p.b_f32, p.b_vec, p.C, 0.f);
  auto col = [&](int i) { return chunk_col<V, NC, kMode>(i); };
  auto have = [&](int i) { return kMode == kExact || col(i) < p.C; };
  T* y = static_cast<T*>(p.y) + walk.row * p.ldy;
  const long long y_step = walk.step * p.ldy;
  bool fail = false;
  int odd = 0;
  for (; walk.more(); walk.next(), y += y_step) {
    fail = !mbar_wait(&full[walk.s], walk.phase, &abort_word, p.timeout_ns, p.status);
    walk.pad();
    Chunk<V> x[ROWS][NC];
    float sum[ROWS], mu[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const uint32_t at = walk.column0(j, 0);
      F2 t = f2(0.f, 0.f);
      mu[j] = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (have(i)) {
          RawChunk<T, V> r;
          r.template load<kMode>(at + static_cast<uint32_t>(col(i)) * static_cast<uint32_t>(sizeof(T)), p.C - col(i));
          x[j][i] = r.values();
        } else {
          x[j][i].zero();
        }
#pragma unroll
        for (int k = 0; k < P; ++k) t = f2_add(t, x[j][i].p[k]);
      }
      sum[j] = f2_sum(t);
    }
    if (layer) {
      cta_sum<ROWS>(sum, red[odd], fail);
      odd ^= 1;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        mu[j] = sum[j] * p.inv_c;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const float m = have(i) ? -mu[j] : 0.f;
          const F2 nm = f2(m, m);
#pragma unroll
          for (int k = 0; k < P; ++k) x[j][i].p[k] = f2_add(x[j][i].p[k], nm);
          if (kMode == kShifted && have(i) && col(i) + V > p.C) {
            asm volatile("" ::: "memory");   // a branch that few warps take, not selects in all
            x[j][i].cut(p.C - col(i));
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      F2 t = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int k = 0; k < P; ++k) t = f2_fma(x[j][i].p[k], x[j][i].p[k], t);
      sum[j] = f2_sum(t);
    }
    cta_sum<ROWS>(sum, red[odd], fail);  // every thread has read the stage; `fail` is now the CTA's
    odd ^= 1;
    if (kMode != kShifted && !fail) walk.refill();
    const int rows = walk.total() - walk.row;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      sum[j] = rsqrtf(sum[j] * p.inv_c + p.eps);   // within 2 ulp, a twentieth of a root and a quotient
      if (p.stats && threadIdx.x == 0 && j < rows) {
        p.stats[walk.row + j] = mu[j];
        p.stats[p.T + walk.row + j] = sum[j];
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (!have(i)) continue;
      const Chunk<V> wc = w.at(i), bc = b.at(i);
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const F2 rr = f2(sum[j], sum[j]);
#pragma unroll
        for (int k = 0; k < P; ++k) x[j][i].p[k] = f2_fma(f2_mul(x[j][i].p[k], rr), wc.p[k], bc.p[k]);
        if (kMode != kShifted && j < rows) store_chunk<T, V>(y + j * p.ldy, x[j][i], col(i));
      }
    }
    if constexpr (kMode == kShifted) {
      T* yr = y;
#pragma unroll
      for (int j = 0; j < ROWS; ++j, yr += p.ldy) {
        ShiftedStore<T, V, NC, kMode> shifted(yr);
#pragma unroll
        for (int i = 0; i < NC; ++i) shifted.put(x[j][i], i, p.C, j < rows && have(i));
      }
    }
    if (fail) break;
    if (kMode == kShifted) walk.refill();                // here the rows' registers are free
  }
  if (fail) walk.settle();
}

// Rows too long for the registers of 512 threads: three passes over the row.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_fwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[64];
  bool none = false;
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
      cta_sum<1>(s, red, none);
      mu = s[0] * p.inv_c;
    }
    float ss[1] = {0.f};
    for (int c = threadIdx.x; c < p.C; c += kMaxThreads) {
      v.load(xr + c);
      ss[0] = fmaf(v.at(0) - mu, v.at(0) - mu, ss[0]);
    }
    cta_sum<1>(ss, red + 32, none);
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

// Backward, ROWS rows of a CTA per turn; NC chunks a thread.  Between the sums and dx a thread keeps
// xh and h of its columns, or (kRaw, where those and dw, db would not fit its registers) the raw
// elements, and forms them again.
template <typename T, int V, int NC, int ROWS, bool kRaw, int kHeld, int kRegs, int kMode>
__global__ void __launch_bounds__(kMaxThreads) __maxnreg__(kRegs) norm_bwd_kernel(const NormParams p, const bool layer) {
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ float red[2][16 * 2 * ROWS];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_word;
  constexpr int P = Chunk<V>::kPairs;
  Walk<T, kMode, ROWS, 2> walk(p, ring_mem, full);
  walk.begin(&abort_word);
  if (threadIdx.x == 0) grid_launch_dependents();     // the column sums' second kernel may take its place
  auto col = [&](int i) { return chunk_col<V, NC, kMode>(i); };
  auto have = [&](int i) { return kMode == kExact || col(i) < p.C; };
  const Held<V, NC, kHeld, kMode> wh(p.w, p.w_f32, p.w_vec, p.C, 1.f);
  Chunk<V> dw[NC], db[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    dw[i].zero();
    db[i].zero();
  }
  T* y = static_cast<T*>(p.y) + (p.y ? walk.row * p.ldy : 0);
  const long long y_step = walk.step * p.ldy;
  bool fail = false;
  int odd = 0;
  // the rows' mu and r, read a turn ahead; a padded row's r is zero, so that it adds nothing
  float mu_n[ROWS], r_n[ROWS];
  auto stats_of = [&](int row0) {
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int t = min(row0 + j, walk.total() - 1);
      mu_n[j] = layer ? __ldg(p.stats + t) : 0.f;
      r_n[j] = __ldg(p.stats + p.T + t);
      if (row0 + j >= walk.total()) mu_n[j] = r_n[j] = 0.f;
    }
  };
  stats_of(walk.row);
  for (; walk.more(); walk.next(), odd ^= 1, y += y_step) {
    float mu[ROWS], r[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      mu[j] = mu_n[j];
      r[j] = r_n[j];
    }
    fail = !mbar_wait(&full[walk.s], walk.phase, &abort_word, p.timeout_ns, p.status);
    walk.pad();
    Chunk<V> x[ROWS][kRaw ? 1 : NC], h[ROWS][kRaw ? 1 : NC];     // xh and dy w
    RawChunk<T, V> rx[ROWS][kRaw ? NC : 1], rg[ROWS][kRaw ? NC : 1];
    float sums[2 * ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const uint32_t ax = walk.column0(j, 0), ag = walk.column0(j, 1);
      const F2 nm = f2(-mu[j], -mu[j]), rr = f2(r[j], r[j]);
      F2 s1 = f2(0.f, 0.f), s2 = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (!have(i)) continue;
        const Chunk<V> w = wh.at(i);
        RawChunk<T, V> a, g;
        const uint32_t at = static_cast<uint32_t>(col(i)) * static_cast<uint32_t>(sizeof(T));
        a.template load<kMode>(ax + at, p.C - col(i));
        g.template load<kMode>(ag + at, p.C - col(i));
        if (kRaw) {
          rx[j][kRaw ? i : 0] = a;
          rg[j][kRaw ? i : 0] = g;
        }
        Chunk<V> xh = a.values(), hh = g.values();
#pragma unroll
        for (int k = 0; k < P; ++k) {
          xh.p[k] = f2_mul(f2_add(xh.p[k], nm), rr);
          dw[i].p[k] = f2_fma(hh.p[k], xh.p[k], dw[i].p[k]);
          db[i].p[k] = f2_add(db[i].p[k], hh.p[k]);
          hh.p[k] = f2_mul(hh.p[k], w.p[k]);
          s1 = f2_add(s1, hh.p[k]);
          s2 = f2_fma(hh.p[k], xh.p[k], s2);
        }
        if (!kRaw) {
          x[j][kRaw ? 0 : i] = xh;
          h[j][kRaw ? 0 : i] = hh;
        }
      }
      sums[2 * j] = f2_sum(s1);
      sums[2 * j + 1] = f2_sum(s2);
    }
    cta_sum<2 * ROWS>(sums, red[odd], fail);   // every thread has read the stage; `fail` is the CTA's
    if (kMode != kShifted && !fail) walk.refill();
    if (walk.total() - walk.row > walk.step) stats_of(walk.row + walk.step);
    if (p.y) {
      const int rows = walk.total() - walk.row;
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        const float m1 = layer ? sums[2 * j] * p.inv_c : 0.f, m2 = sums[2 * j + 1] * p.inv_c;
        const F2 a = f2(-m1, -m1), b = f2(-m2, -m2), rr = f2(r[j], r[j]), nm = f2(-mu[j], -mu[j]);
        ShiftedStore<T, V, NC, kMode> shifted(y + j * p.ldy);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (kMode != kShifted && !have(i)) continue;
          Chunk<V> xh, hh;
          if (kMode == kShifted && !have(i)) {
            xh.zero();
            hh.zero();
          } else if (kRaw) {
            xh = rx[j][kRaw ? i : 0].values();
            hh = rg[j][kRaw ? i : 0].values();
            const Chunk<V> w = wh.at(i);
#pragma unroll
            for (int k = 0; k < P; ++k) {
              xh.p[k] = f2_mul(f2_add(xh.p[k], nm), rr);
              hh.p[k] = f2_mul(hh.p[k], w.p[k]);
            }
          } else {
            xh = x[j][kRaw ? 0 : i];
            hh = h[j][kRaw ? 0 : i];
          }
#pragma unroll
          for (int k = 0; k < P; ++k) xh.p[k] = f2_mul(f2_fma(xh.p[k], b, f2_add(hh.p[k], a)), rr);
          if constexpr (kMode == kShifted) shifted.put(xh, i, p.C, j < rows && have(i));
          else if (j < rows) store_chunk<T, V>(y + j * p.ldy, xh, col(i));
        }
      }
    }
    if (fail) break;
    if (kMode == kShifted) walk.refill();                // here the rows' registers are free
  }
  if (fail) walk.settle();
  if (!p.part) return;
  float* out = p.part + static_cast<long long>(blockIdx.x) * 2 * p.C;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (!have(i)) continue;
    store_sums<V>(out, dw[i], col(i), p.C);
    store_sums<V>(out + p.C, db[i], col(i), p.C);
  }
}

// Rows too long for registers: sums of a row from two passes; a thread's columns are strided
// by 512, its dw and db kept in the CTA's own workspace row (each element touched by one
// thread only).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_long_kernel(const NormParams p, const bool layer) {
  __shared__ float red[32];
  bool none = false;
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
      cta_sum<2>(s, red, none);
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

// dw, db [C] from the CTAs' partial rows: 8 columns a block (one sector of a row), a thread every 64th row
// of a column, eight loads at a time, joined in order.  Launched beside the backward (its blocks wait
// for it to finish).
constexpr int kFinishCols = 8;
__global__ void __launch_bounds__(512) norm_finish_kernel(const float* part, int n, int C, float* dw, float* db) {
  constexpr int kRows = 512 / kFinishCols;
  __shared__ float sh[kRows][kFinishCols + 1];
  const int col = threadIdx.x % kFinishCols, sub = threadIdx.x / kFinishCols;
  const int c = blockIdx.x * kFinishCols + col;
  float* out = blockIdx.y ? db : dw;
  grid_dependency_wait();
  if (!out) return;
  const float* q = part + static_cast<long long>(blockIdx.y) * C + c;
  float s = 0.f;
  if (c < C) {
    for (int i0 = sub; i0 < n; i0 += kRows * 8) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = i0 + kRows * k < n ? q[static_cast<long long>(i0 + kRows * k) * 2 * C] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  }
  sh[sub][col] = s;
  __syncthreads();
  if (threadIdx.x >= 4 * kFinishCols) return;          // four threads a column, then one
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < kRows / 4; ++i) t += sh[sub * (kRows / 4) + i][col];
  t += __shfl_xor_sync(0xffffffffu, t, kFinishCols);
  t += __shfl_xor_sync(0xffffffffu, t, 2 * kFinishCols);
  if (sub == 0 && c < C) out[c] = t;
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
         v->rows * v->cols == C && one_piece(*v);
}

// How a row length is worked on: vectors (or single elements) per thread (0: the long form), rows
// per turn, threads, registers a thread, CTAs per SM, ring stages and bytes of a row's slot.
struct Form {
  int nv, rows, threads, regs, per_sm, stages, slot;
};

// Threads that share a row: each holds nv vectors of it, a whole number of warps in all.
int row_threads(long long vectors, int nv) {
  return static_cast<int>(((vectors + nv - 1) / nv + 31) / 32 * 32);
}

// The ring of a form: as many CTAs per SM as its registers allow (each of the four schedulers has 16384,
// so 104 and 112 a thread allow no more warps than 128; at most 16 CTAs), the stages that then fit
// their shared memory, at most kMaxStages; fewer CTAs when two stages do not.  A CTA too many would
// run after the others, with none beside it.
bool ring_form(Form* f, long long C, bool f32, bool vec, int ops) {
  const int size = f32 ? 4 : 2;
  f->slot = static_cast<int>((C * size + 15) / 16 * 16 + (vec ? 0 : 16));
  const size_t stage = static_cast<size_t>(f->rows) * ops * f->slot;
  f->per_sm = 16384 / (32 * f->regs) * 4 / (f->threads / 32);
  if (f->per_sm > 16) f->per_sm = 16;
  if (f->per_sm < 1) f->per_sm = 1;
  for (;; --f->per_sm) {
    const size_t room = static_cast<size_t>(kSmemPerSm) / f->per_sm - 2048;
    f->stages = static_cast<int>(room / stage < kMaxStages ? room / stage : kMaxStages);
    if (f->stages >= 2 || f->per_sm == 1) break;
  }
  return f->stages >= 2;
}

// A form that takes nv vectors a thread and up to `top` threads; worth: its rate beside the first one's
// where both fill the schedulers (it has fewer rows a turn to spread the turn's waits over, or spills).
struct Option {
  int nv, rows, top, regs;
  double worth;
};

// The form with the most of the schedulers' warps at work: lanes that have columns, times the warps that
// the CTAs on an SM occupy of 16, times its worth; a CTA alone on its SM has nothing to run while its
// rows' sums meet, and counts four fifths; one warp needs no CTA barrier, which is a gain where rows are
// shifted (60000 x 509 bf16 backward 78 us with two warps, 70 with one).  Backward, 32760 rows of bf16:
// 2560 columns took 124 us with ten warps of 8 elements a thread and 90 with five of 16, 1280 columns 52
// and 60, 4096 columns 155 and 138.
template <int kOptions>
Form pick_form(const Option (&options)[kOptions], long long C, bool f32, bool vec, int ops) {
  const long long n = (C + (f32 ? 3 : 7)) / (f32 ? 4 : 8);
  Form best{0, 1, kMaxThreads, 64, 2, 0, 0};
  if (C > (1 << 20)) return best;
  double most = 0;
  for (const Option& q : options) {
    if (n > static_cast<long long>(q.nv) * q.top) continue;
    Form f{q.nv, q.rows, row_threads(n, q.nv), q.regs, 0, 0, 0};
    if (!ring_form(&f, C, f32, vec, ops)) continue;
    const double rate = static_cast<double>(n) / (q.nv * f.threads) * (f.per_sm * f.threads) / 512 * q.worth *
                        (f.per_sm == 1 ? 0.8 : f.threads == 32 && !vec ? 1.3 : 1);
    if (rate > most) {
      most = rate;
      best = f;
    }
  }
  return best;
}

// Forward: 8 elements a thread (rows of up to 32 vectors, one warp; two warps of it took 27 us for 60000 x
// 512 bf16 where one of 16 elements takes 21), 16 and four rows a turn, or more and fewer rows.  Aligned rows
// wait for memory whatever the warps and take the first form that holds them (8192 columns of bf16 took
// 159 us with 16 warps of 16 elements and 190 with 8 of 32); shifted ones are bound by instructions (4099
// columns of bf16 260 us with nine warps of 16, 212 with five of 32).
Form fwd_form(long long C, bool f32, bool vec) {
  const Option first[] = {{1, 4, 32, 104, 1}, {2, 4, 512, 128, 0.1}, {4, 2, 512, 128, 0.01}, {8, 1, 512, 128, 0.001}},
               shifted[] = {{1, 4, 32, 104, 1}, {2, 4, 512, 128, 1}, {4, 2, 512, 128, 0.75}, {8, 1, 512, 128, 0.3}};
  return vec ? pick_form(first, C, f32, true, 1) : pick_form(shifted, C, f32, false, 1);
}

// Backward: 8 elements a thread and four rows a turn (its dw, db, weight, xh and h take registers
// each), 16 and two, 24 or 32 and one; shifted rows half as many rows a turn.  (24: 6144 columns of bf16
// 242 to 220 us, 12001 columns 1037 to 874.)
Form bwd_form(long long C, bool f32, bool vec) {
  const int h = vec ? 1 : 2;
  const Option v8[] = {{1, 4 / h, 512, 128, 1}, {2, 2 / h, 512, 128, 0.9}, {3, 1, 512, 128, vec ? 0.8 : 0.65},
                       {4, 1, 512, 128, vec ? 0.45 : 0.6}},
               v4[] = {{2, 4 / h, 512, 128, 1}, {4, 2 / h, 512, 128, 0.75}, {8, 1, 512, 128, 0.4}};
  return f32 ? pick_form(v4, C, true, vec, 2) : pick_form(v8, C, false, vec, 2);
}

template <typename K>
int launch(K kernel, int blocks, const Form& f, size_t smem, const NormParams& p, bool layer, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
  if (e == cudaSuccess) {
    kernel<<<blocks, f.threads, smem, st>>>(p, layer);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

int blocks_of(long long T, const Form& f) {
  const long long need = (T + f.rows - 1) / f.rows, cap = static_cast<long long>(f.per_sm) * device_sm_count();
  return static_cast<int>(need < cap ? need : cap);
}

template <typename T>
int dispatch_fwd(NormParams p, bool vec, bool layer, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const Form f = fwd_form(p.C, sizeof(T) == 4, vec);
  if (f.nv == 0) {
    const long long cap = 4ll * device_sm_count();
    norm_fwd_long_kernel<T><<<static_cast<unsigned>(p.T < cap ? p.T : cap), kMaxThreads, 0, st>>>(p, layer);
    return last_launch();
  }
  p.stages = f.stages;
  p.slot = f.slot;
  const size_t smem = static_cast<size_t>(f.stages) * f.rows * f.slot;
  const int g = blocks_of(p.T, f);
  const bool exact = vec && p.C == f.nv * f.threads * V;
  const bool packed = (!p.w || (!p.w_f32 && p.w_vec)) && (!p.b || (!p.b_f32 && p.b_vec));
  const int mode = !vec ? kShifted : exact ? kExact : kWhole;
#define WP_FWD(...) \
  (mode == kExact ? launch(norm_fwd_kernel<T, V, __VA_ARGS__, kExact>, g, f, smem, p, layer, st) \
   : mode == kWhole ? launch(norm_fwd_kernel<T, V, __VA_ARGS__, kWhole>, g, f, smem, p, layer, st) \
                    : launch(norm_fwd_kernel<T, V, __VA_ARGS__, kShifted>, g, f, smem, p, layer, st))
  switch (f.nv) {
    case 1: return WP_FWD(1, 4, kHeldValues, 104);
    case 2:
      if constexpr (V == 4) return WP_FWD(2, 4, kHeldValues, 112);
      else return packed ? WP_FWD(2, 4, kHeldPacked, 128) : WP_FWD(2, 4, kHeldNot, 128);
    case 4:
      if constexpr (V == 4) return WP_FWD(4, 2, kHeldValues, 128);
      else return packed ? WP_FWD(4, 2, kHeldPacked, 128) : WP_FWD(4, 2, kHeldNot, 128);
    default: return WP_FWD(8, 1, kHeldNot, 128);
  }
#undef WP_FWD
}

template <typename T>
int dispatch_bwd(NormParams p, bool vec, bool layer, int* grid, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const Form f = bwd_form(p.C, sizeof(T) == 4, vec);
  const int g = *grid = blocks_of(p.T, f);
  if (f.nv == 0) {
    norm_bwd_long_kernel<T><<<g, kMaxThreads, 0, st>>>(p, layer);
    return last_launch();
  }
  p.stages = f.stages;
  p.slot = f.slot;
  const size_t smem = static_cast<size_t>(f.stages) * f.rows * 2 * f.slot;
  const bool exact = vec && p.C == f.nv * f.threads * V;
  const bool packed = !p.w || (!p.w_f32 && p.w_vec);
  const int mode = !vec ? kShifted : exact ? kExact : kWhole;
#define WP_BWD(NC, ROWS, RAW, HELD)                                                                                 \
  (mode == kExact   ? launch(norm_bwd_kernel<T, V, NC, ROWS, RAW, HELD, 128, kExact>, g, f, smem, p, layer, st)     \
   : mode == kWhole ? launch(norm_bwd_kernel<T, V, NC, ROWS, RAW, HELD, 128, kWhole>, g, f, smem, p, layer, st)     \
                    : launch(norm_bwd_kernel<T, V, NC, (ROWS + 1) / 2, RAW, HELD, 128, kShifted>, g, f, smem, p, layer, st))
  if constexpr (V == 8) {
    switch (f.nv) {
      case 1: return WP_BWD(1, 4, false, kHeldValues);
      case 2: return packed ? WP_BWD(2, 2, false, kHeldPacked) : WP_BWD(2, 2, false, kHeldNot);
      case 3: return packed ? WP_BWD(3, 1, true, kHeldPacked) : WP_BWD(3, 1, true, kHeldNot);
      default: return packed ? WP_BWD(4, 1, true, kHeldPacked) : WP_BWD(4, 1, true, kHeldNot);
    }
  } else {
    switch (f.nv) {
      case 2: return WP_BWD(2, 4, false, kHeldValues);
      case 4: return WP_BWD(4, 2, false, kHeldValues);
      default: return WP_BWD(8, 1, false, kHeldNot);
    }
  }
#undef WP_BWD
}

bool valid_rows(const wp_mat* m) {
  return m && m->rows >= 0 && m->cols > 0 && (m->data || m->rows == 0) && m->ld >= m->cols &&
         (m->dtype == WP_BF16 || m->dtype == WP_FP32);
}

}  // namespace

size_t norm_bwd_workspace(long long T, long long C, bool f32) {
  // a partial row of dw and db for each CTA of either form (16-byte aligned rows or not)
  if (T < 0 || C <= 0) return 0;
  int n = blocks_of(T, bwd_form(C, f32, false));
  if (C % (f32 ? 4 : 8) == 0) {
    const int v = blocks_of(T, bwd_form(C, f32, true));
    if (v > n) n = v;
  }
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
  if (!aligned_element(X->data, X->dtype) || !aligned_element(Y->data, Y->dtype) || !aligned_element(stats, WP_FP32) ||
      (weight && !aligned_element(weight->data, weight->dtype)) || (bias && !aligned_element(bias->data, bias->dtype)))
    return WP_ERR_ALIGN;
  if (X->cols > 0x3FFFFFFFLL || X->rows > 0x7FFFFFFFLL) return WP_ERR_UNSUPPORTED;
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
  p.timeout_ns = device_wait_limit_ns();
  p.status = tc_status_ptr();
  if (!p.status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
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
    if (o->rows * o->cols != X->cols || !one_piece(*o)) return WP_ERR_SHAPE;
    if (!aligned_element(o->data, WP_FP32)) return WP_ERR_ALIGN;
  }
  if (!aligned_element(X->data, X->dtype) || !aligned_element(dY->data, dY->dtype) || !aligned_element(stats, WP_FP32) ||
      (dX && !aligned_element(dX->data, dX->dtype)) || (weight && !aligned_element(weight->data, weight->dtype)))
    return WP_ERR_ALIGN;
  if (X->cols > 0x3FFFFFFFLL || X->rows > 0x7FFFFFFFLL) return WP_ERR_UNSUPPORTED;
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
  p.timeout_ns = device_wait_limit_ns();
  p.status = tc_status_ptr();
  if (!p.status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
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
  cfg.gridDim = dim3((p.C + kFinishCols - 1) / kFinishCols, 2);
  cfg.blockDim = dim3(512);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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
