// wp_multi_term.cuh -- the adapters' term of a tile of rows with a slot each: s_t (X[t] A^T) B^T from
// H~ and the slots' columns of B, in mma.sync fragments straight from global memory (shared by
// the kernels for a few rows).
#pragma once

#include <cstdint>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

__device__ __forceinline__ float bf2f(uint32_t h) { return __uint_as_float(h << 16); }

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// D[16 x 8] += A[16 x 16] B[16 x 8], bf16 inputs, fp32 sums
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kTermRows = 128;

struct TermShared {
  int act[kTermRows];                                // the rows' slots (-1: no adapter)
  int g_slot[kTermRows], g_of[kTermRows], g_count[4];  // groups of up to 8 rows of one slot
  __align__(8) uint8_t g_row[kTermRows][8];
};

// Up to 16 rows, most with a slot of their own, of rank 8 or 16: an mma.sync would use one row of its eight,
// and its chain H~, products, next groups is what the rest of the kernel waits for.  A thread takes a
// column and every other row; all of its B is on its way to registers before H~ is waited for, and H~
// comes to shared memory (in delta's place) at once.  64 rows of 64 slots of rank 16 beside 5120 -> 5120:
// 21.4 us by groups, 19.7 so; 16 rows of 16 beside the 4-bit 4096 -> 28672 39.7 and 36.9.  At
// larger ranks a column's B no longer comes in one piece: 16 rows of rank 64 25 and 34.5.
constexpr int kTermSingles = 8;                      // rows a thread
__device__ __forceinline__ void singles_term(const MultiCall& c, const TermShared& sh, float* delta, int first, int cnt,
                                             int n0, int c0, int wide, int tid) {
  const int col = tid & 127, n = min(n0 + col, c.N - 1);
  auto load = [&](int r, uint4 (&v)[kTermSingles]) {
#pragma unroll
    for (int k = 0; k < kTermSingles; ++k) {
      const int i = (tid >> 7) + 2 * k, a = i < cnt && r < c.R ? sh.act[i] : -1;
      v[k] = a >= 0 ? ldg16(c.B + (static_cast<long long>(a) * c.N + n) * c.R + r) : make_uint4(0, 0, 0, 0);
    }
  };
  uint4 b0[kTermSingles], b1[kTermSingles];
  load(0, b0);
  load(8, b1);
  grid_dependency_wait();
  uint16_t* h = reinterpret_cast<uint16_t*>(delta);  // [cnt][wide]
  const int pieces = wide / 8;
  for (int p = tid; p < cnt * pieces; p += 256) {
    const int i = p / pieces, o = (p - i * pieces) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (sh.act[i] >= 0)
      v = *reinterpret_cast<const uint4*>(c.H + (static_cast<long long>(first + i) * c.G + c0) * c.R16 + o);
    *reinterpret_cast<uint4*>(h + i * wide + o) = v;
  }
  named_bar_sync(1, 256);
  F2 sum[kTermSingles];
#pragma unroll
  for (int k = 0; k < kTermSingles; ++k) sum[k] = f2(0.f, 0.f);
  const uint16_t* hg = h + (n / c.og - c0) * c.R16;
  auto add = [&](int r, const uint4 (&v)[kTermSingles]) {
    if (r >= c.R) return;
#pragma unroll
    for (int k = 0; k < kTermSingles; ++k) {
      const int i = (tid >> 7) + 2 * k;
      if (i >= cnt) continue;
      const uint4 q = *reinterpret_cast<const uint4*>(hg + i * wide + r);
      const uint32_t hw[4] = {q.x, q.y, q.z, q.w}, bw[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[k] = f2_fma(f2(__uint_as_float(hw[e] << 16), __uint_as_float(hw[e] & 0xffff0000u)),
                        f2(__uint_as_float(bw[e] << 16), __uint_as_float(bw[e] & 0xffff0000u)), sum[k]);
    }
  };
  add(0, b0);
  add(8, b1);
  named_bar_sync(1, 256);                            // H~ has been read
#pragma unroll
  for (int k = 0; k < kTermSingles; ++k) {
    float x, y;
    f2_get(sum[k], x, y);
    const int i = (tid >> 7) + 2 * k;
    if (i < cnt) delta[i * 128 + col] = x + y;
  }
}

// delta[i][128 columns from n0] of the cnt (<= kTermRows) rows from `first` on, by 256 threads (tid; named
// barrier 1), 16 columns a warp.  The slots and scales are inputs, so only H~ waits for the kernel before
// (whose end every thread has waited for on return).  The caller passes a barrier before it
// reads delta.
__device__ __forceinline__ void adapters_term(const MultiCall& c, TermShared& sh, float* delta, int first, int cnt, int n0,
                                              int tid) {
  const int lane = tid & 31, w8 = tid >> 5;
  // the share's rows in groups of up to 8 rows of one slot (the slots and scales are inputs: this
  // runs beside the kernel that forms H~)
  int a = -1;
  if (tid < cnt) {
    const int t = first + tid;
    a = c.slot[t];
    if (a < 0 || a >= c.S) {
      a = -1;
    } else {
      float s = c.scale[a];
      if (c.row_scale) s = __fmul_rn(s, c.row_scale[t]);
      if (__fmul_rn(s, c.request_scale) == 0.f) a = -1;
    }
    sh.act[tid] = a;
  }
  named_bar_sync(1, 256);
  int before = 0, lead = tid;                       // rows of this slot before this one; its group's first
  if (a >= 0)
    for (int j = 0; j < tid; ++j)
      if (sh.act[j] == a) {
        if ((before & 7) == 0) lead = j;
        ++before;
      }
  if ((before & 7) == 0) lead = tid;
  const bool leads = a >= 0 && lead == tid;
  const uint32_t firsts = __ballot_sync(0xffffffffu, leads);
  if (lane == 0 && w8 < 4) sh.g_count[w8] = __popc(firsts);
  named_bar_sync(1, 256);
  int ng = 0, gid = __popc(firsts & ((1u << lane) - 1));
  for (int w = 0; w < 4; ++w) {
    if (w < w8) gid += sh.g_count[w];
    ng += sh.g_count[w];
  }
  const int c0 = n0 / c.og, wide = (min(n0 + 127, c.N - 1) / c.og - c0 + 1) * c.R16;
  if (c.R <= 16 && cnt <= 2 * kTermSingles && cnt <= 2 * ng && wide <= 256) {
    singles_term(c, sh, delta, first, cnt, n0, c0, wide, tid);
    return;
  }
  if (leads) {
    sh.g_slot[gid] = a;
    sh.g_of[tid] = gid;
    *reinterpret_cast<uint2*>(sh.g_row[gid]) = make_uint2(0xffffffffu, 0xffffffffu);
  }
  named_bar_sync(1, 256);
  if (a >= 0) sh.g_row[sh.g_of[lead]][before & 7] = static_cast<uint8_t>(tid);
  for (int i = tid >> 7; i < cnt; i += 2)
    if (sh.act[i] < 0) delta[i * 128 + (tid & 127)] = 0.f;
  named_bar_sync(1, 256);
  // this warp's 16 output columns; the two halves may lie in different column groups
  const int nw = n0 + w8 * 16;
  const int n_lo = min(nw + (lane >> 2), c.N - 1), n_hi = min(nw + 8 + (lane >> 2), c.N - 1);
  const int c_lo = min(nw, c.N - 1) / c.og, c_hi = min(nw + 8, c.N - 1) / c.og;
  const int kl = (lane & 3) * 8;
  const int hld = c.G * c.R16;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int g = 0; g < ng; ++g) {                    // pull the slots' columns of B toward L2 meanwhile
    const uint16_t* b = c.B + (static_cast<long long>(sh.g_slot[g]) * c.N + min(nw + (lane & 15), c.N - 1)) * c.R;
    for (int o = (lane >> 4) * 64; o < c.R; o += 128) prefetch_l2(b + o);
  }
  // Groups whose loads are issued together; the first ones' columns of B before the wait for H~.
  constexpr int U = 4;
  bool waited = false;
  for (int g0 = 0; g0 < ng; g0 += U) {
    float d[U][4], e[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) d[u][k] = e[u][k] = 0.f;
    for (int q = 0; q < c.R; q += 32) {             // the whole warp: lanes past the rank add zeros
      const int r = q + kl;
      const bool ok = r < c.R;
      uint4 lo[U], hi[U], h[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long sl = static_cast<long long>(sh.g_slot[min(g0 + u, ng - 1)]) * c.N;
        lo[u] = ok ? ldg16(c.B + (sl + n_lo) * c.R + r) : zero;
        hi[u] = ok ? ldg16(c.B + (sl + n_hi) * c.R + r) : zero;
      }
      if (!waited) {
        grid_dependency_wait();
        waited = true;
      }
      auto load_h = [&](int cg) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int tr = sh.g_row[min(g0 + u, ng - 1)][lane >> 2];
          h[u] = ok && tr < 255
                     ? *reinterpret_cast<const uint4*>(c.H + static_cast<long long>(first + tr) * hld + cg * c.R16 + r)
                     : zero;
        }
      };
      load_h(c_lo);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        mma_16816(d[u], lo[u].x, hi[u].x, lo[u].y, hi[u].y, h[u].x, h[u].y);
        mma_16816(d[u], lo[u].z, hi[u].z, lo[u].w, hi[u].w, h[u].z, h[u].w);
      }
      if (c_hi != c_lo) {                           // (a warp's two halves in different column groups)
        load_h(c_hi);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          mma_16816(e[u], lo[u].x, hi[u].x, lo[u].y, hi[u].y, h[u].x, h[u].y);
          mma_16816(e[u], lo[u].z, hi[u].z, lo[u].w, hi[u].w, h[u].z, h[u].w);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g0 + u < ng) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int tr = sh.g_row[g0 + u][2 * (lane & 3) + k];
          if (tr < 255) {
            float* o = delta + tr * 128 + w8 * 16 + (lane >> 2);
            o[0] = d[u][k];
            o[8] = c_hi != c_lo ? e[u][2 + k] : d[u][2 + k];
          }
        }
      }
    }
    __syncwarp();
  }
  if (!waited) grid_dependency_wait();
}

}  // namespace wp
