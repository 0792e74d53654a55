// wp_multi_small.cu -- the many-adapter projection for a few rows (decode batches).
//
//   Y[t, g] = X[t] W_g^T + bias_g + s_t (X[t] A_{a,g}^T) B_{a,g}^T,   a = slot[t]
//
// With this few rows every byte of W, and of the A and B of each slot present, is read for a
// handful of products, so HBM is the floor and the start-up of each kernel the next bound.  Two
// kernels, the second started while the first runs (programmatic dependent launch):
//
//   shrink  one CTA per (32 rows of one slot, 16 rank rows): its 8 warps take turns along K with loads
//           straight from global into mma.sync fragments -- the rank rows are the 16-row operand,
//           the slot's rows of X the 8-wide one, both through the same permutation of k so that
//           every lane loads 16 consecutive bytes -- and leave H~ = bf16(s X A^T).  mma.sync
//           rather than tcgen05: there is no tile to keep, a row belongs to one slot only.  bf16, as
//           the operand of the second product (two pieces would double its work): 64 rows of rank 16
//           are 0.3 % further from the 64-bit result than with H~ in fp32, Y's own rounding the rest.
//           (One or two rows of few ranks do without: the main kernel forms their H~ from its part of K.)
//   main    W^T tiles of 128 output columns as the M = 128 operand of tcgen05.mma and the rows of
//           X (rounded up to 16) as its width, W and X by TMA.  K is split over a cluster of up to
//           8 CTAs so that every SM is streaming W from the first moment; while they do, eight more
//           warps form the adapters' term of the CTA's share of the rows, 16 output columns a warp,
//           rows of one slot together up to 8 (the mma.sync fragments again, straight from global
//           memory), and the partial tiles meet through distributed shared memory, added in CTA order.
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_multi_term.cuh"
#include "wp_ptx.cuh"

namespace wp {

namespace {

constexpr int kShrinkThreads = 256;
constexpr int kShrinkWarps = kShrinkThreads / 32;

// H~ of up to 8 NT rows (list[0 .. n)) for 16 rank rows, K split over the warps; the partial
// sums go to red[warp][16][8 NT].  U: 32-wide k steps whose loads are issued together.
template <int NT, int U>
__device__ __forceinline__ void shrink_pass(const MultiCall& c, const uint16_t* a_row0, const uint16_t* a_row1,
                                            const int* list, int n, float* red, int part, int parts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kl = (lane & 3) * 8;                   // this lane's 8 k of every 32
  const uint16_t* x[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int j = i * 8 + (lane >> 2);
    x[i] = c.X + static_cast<long long>(list[j < n ? j : 0]) * c.ldx;
  }
  float d[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) d[i][k] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k0 = (part * kShrinkWarps + warp) * (32 * U); k0 < c.K; k0 += parts * kShrinkWarps * 32 * U) {
    uint4 a0[U], a1[U], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * 32 + kl;
      const bool ok = k < c.K;
      a0[u] = ok ? ldg16(a_row0 + k) : zero;
      a1[u] = ok ? ldg16(a_row1 + k) : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i) b[u][i] = ok ? ldg16(x[i] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        mma_16816(d[i], a0[u].x, a1[u].x, a0[u].y, a1[u].y, b[u][i].x, b[u][i].y);
        mma_16816(d[i], a0[u].z, a1[u].z, a0[u].w, a1[u].w, b[u][i].z, b[u][i].w);
      }
  }
  // d[i][0..1]: rank row lane / 4, X rows 8 i + 2 (lane % 4) + {0, 1}; d[i][2..3]: rank row + 8
  float* out = red + warp * (16 * 8 * NT);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int col = i * 8 + (lane & 3) * 2;
    float* o = out + (lane >> 2) * (8 * NT) + col;
    o[0] = d[i][0];
    o[1] = d[i][1];
    o[8 * 8 * NT] = d[i][2];
    o[8 * 8 * NT + 1] = d[i][3];
  }
}

// Grid: (rows x parts, chunks of 16 rank rows), a cluster of `parts` CTAs per (row, chunk) sharing K.
__global__ void __launch_bounds__(kShrinkThreads) multi_shrink_small_kernel(const MultiCall c, const int parts) {
  __shared__ int list[kMultiFewRows];
  __shared__ int wcount[kShrinkWarps];
  __shared__ float red[kShrinkWarps * 16 * 32];
  __shared__ float sums[16 * 32];
  const int t = static_cast<int>(blockIdx.x) / parts, chunk = blockIdx.y;
  const int part = parts > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  const int a = c.slot[t];
  if (a < 0 || a >= c.S) return;                     // the same in every CTA of the cluster
  // the rows of this slot in order, 32 to a pass; the first of each pass stands for it
  int before = 0, n = 0;
  for (int base = 0; base < c.T; base += kShrinkThreads) {
    const int j = base + tid;
    const bool mine = j < c.T && c.slot[j] == a;
    const uint32_t m = __ballot_sync(0xffffffffu, mine), em = __ballot_sync(0xffffffffu, mine && j < t);
    if (lane == 0) wcount[warp] = __popc(m) | __popc(em) << 16;
    __syncthreads();
    int at = n;                                      // this slot's rows before this warp's
    for (int w = 0; w < kShrinkWarps; ++w) {
      if (w < warp) at += wcount[w] & 0xffff;
      n += wcount[w] & 0xffff;
      before += wcount[w] >> 16;
    }
    if (mine) list[at + __popc(m & ((1u << lane) - 1))] = j;
    __syncthreads();
  }
  if (before % 32) return;                           // the same in every CTA of the cluster
  n = min(n - before, 32);
  const int rows = c.G * c.R;
  const int j0 = chunk * 16;
  const uint16_t* A = c.A + static_cast<long long>(a) * rows * c.K;
  // rank rows past the last repeat it; their sums are not kept
  const uint16_t* a_row0 = A + static_cast<long long>(min(j0 + (lane >> 2), rows - 1)) * c.K;
  const uint16_t* a_row1 = A + static_cast<long long>(min(j0 + 8 + (lane >> 2), rows - 1)) * c.K;
  const float sa = c.scale[a];
  const int nt = n <= 8 ? 1 : 4;
  if (nt == 1) shrink_pass<1, 4>(c, a_row0, a_row1, list + before, n, red, part, parts);
  else shrink_pass<4, 2>(c, a_row0, a_row1, list + before, n, red, part, parts);
  __syncthreads();
  for (int i = tid; i < 16 * n; i += kShrinkThreads) {
    const int r = i / n, col = i - r * n;              // rank row of the chunk, row of the pass
    float h = 0.f;
#pragma unroll
    for (int w = 0; w < kShrinkWarps; ++w) h += red[(w * 16 + r) * (8 * nt) + col];
    sums[r * 32 + col] = h;
  }
  __syncthreads();
  if (parts > 1) cluster_sync();                       // every CTA's share of K is summed
  if (part == 0) {
    for (int i = tid; i < 16 * n; i += kShrinkThreads) {
      const int r = i / n, col = i - r * n;
      const int j = j0 + r;
      if (j < rows) {
        float h = sums[r * 32 + col];
        for (int q = 1; q < parts; ++q) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v) : "r"(mapa_shared(smem_u32(&sums[r * 32 + col]), static_cast<uint32_t>(q))));
          h += v;
        }
        const int tt = list[before + col];
        float s = sa;
        if (c.row_scale) s = __fmul_rn(s, c.row_scale[tt]);
        s = __fmul_rn(s, c.request_scale);
        const int g = j / c.R, rr = j - g * c.R;
        uint16_t* out = c.H + static_cast<long long>(tt) * c.G * c.R16 + g * c.R16 + rr;
        uint16_t hb;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(hb) : "f"(h * s));
        *out = hb;
        if (c.R != c.R16 && rr >= c.R - 8) out[8] = 0;   // the group's padding columns
      }
    }
  }
  __syncthreads();
  if (parts > 1) cluster_sync();                       // no CTA leaves while its sums are read
}

// ------------------------------------------------------------------------------ main
struct SmallMaps {
  CUtensorMap x, w;            // boxes of 64 K x t16 rows / 128 rows, 128-byte swizzle
};

constexpr int kSmallThreads = 320;         // warp 0 TMA, warp 1 MMA, warps 2..9 the adapters' term and the output
constexpr int kSmallSmem = 109 * 1024;     // two CTAs per SM, 3 KiB of static arrays each beside it
constexpr int kSmallMaxStages = 8;

struct SmallParams {
  MultiCall c;
  int has_w;
  int tile;                    // rows of X per tile (128, or 64 where shared memory holds no more)
  int t16;                     // MMA width: rows of a tile rounded up to 16
  int splits, kb_per, k_blocks;
  int share;                   // rows of the tile whose output a CTA of the cluster writes
  int stages, stage_bytes;
  uint32_t tmem_cols;
};

// The adapters' term of all of a few rows from this CTA's part of K, [c.T][128] in delta: h (the rows' rank
// values over k0 .. k1, fp32) and then h B^T.  By 256 threads (tid), four rank rows a warp at a time.  The
// parts' terms are added with their products of W, so H~ is never whole and is not rounded.
__device__ __forceinline__ void whole_term(const MultiCall& c, float* delta, int n0, int k0, int k1, int tid) {
  const int lane = tid & 31, w8 = tid >> 5;
  const int ga = n0 / c.og, gb = min(n0 + 127, c.N - 1) / c.og;
  const int nj = (gb - ga + 1) * c.R, rows = c.G * c.R;
  float* h = delta + c.T * 128;                      // [c.T][nj]
  auto slot_of = [&](int t, float& s) {
    int a = c.slot[t];
    s = 0.f;
    if (a < 0 || a >= c.S) return -1;
    s = c.scale[a];
    if (c.row_scale) s = __fmul_rn(s, c.row_scale[t]);
    s = __fmul_rn(s, c.request_scale);
    return s != 0.f ? a : -1;
  };
  const int n = n0 + (tid & 127);
  float s;
  for (int t = tid >> 7; t < c.T && n < c.N; t += 2) {
    const int a = slot_of(t, s);
    if (a >= 0) prefetch_l2(c.B + (static_cast<long long>(a) * c.N + n) * c.R);
  }
  const int quads = nj / 4;
  for (int t = 0; t < c.T; ++t) {
    const int a = slot_of(t, s);
    if (a < 0) continue;
    const uint16_t* x = c.X + t * c.ldx;
    for (int q = w8; q < quads; q += 8) {
      const uint16_t* A = c.A + (static_cast<long long>(a) * rows + ga * c.R + q * 4) * c.K;
      F2 sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = f2(0.f, 0.f);
      for (int k = k0 + lane * 8; k < k1; k += 256) {
        const uint4 xv = ldg16(x + k);
        uint4 av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = ldg16(A + static_cast<long long>(i) * c.K + k);
        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t aw[4] = {av[i].x, av[i].y, av[i].z, av[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sum[i] = f2_fma(f2(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xffff0000u)),
                            f2(__uint_as_float(aw[e] << 16), __uint_as_float(aw[e] & 0xffff0000u)), sum[i]);
        }
      }
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float a0, a1;
        f2_get(sum[i], a0, a1);
        v[i] = a0 + a1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
      if (lane == 0) *reinterpret_cast<float4*>(h + t * nj + q * 4) = make_float4(v[0] * s, v[1] * s, v[2] * s, v[3] * s);
    }
  }
  named_bar_sync(1, 256);
  for (int t = tid >> 7; t < c.T; t += 2) {
    const int a = slot_of(t, s);
    float v = 0.f;
    if (a >= 0 && n < c.N) {
      const uint16_t* b = c.B + (static_cast<long long>(a) * c.N + n) * c.R;
      const float* hg = h + t * nj + (n / c.og - ga) * c.R;
#pragma unroll 4
      for (int r = 0; r < c.R; r += 8) {
        const uint4 bv = ldg16(b + r);
        const float4 h0 = *reinterpret_cast<const float4*>(hg + r), h1 = *reinterpret_cast<const float4*>(hg + r + 4);
        v = fmaf(h0.x, __uint_as_float(bv.x << 16), v);
        v = fmaf(h0.y, __uint_as_float(bv.x & 0xffff0000u), v);
        v = fmaf(h0.z, __uint_as_float(bv.y << 16), v);
        v = fmaf(h0.w, __uint_as_float(bv.y & 0xffff0000u), v);
        v = fmaf(h1.x, __uint_as_float(bv.z << 16), v);
        v = fmaf(h1.y, __uint_as_float(bv.z & 0xffff0000u), v);
        v = fmaf(h1.z, __uint_as_float(bv.w << 16), v);
        v = fmaf(h1.w, __uint_as_float(bv.w & 0xffff0000u), v);
      }
    }
    delta[t * 128 + (tid & 127)] = v;
  }
  named_bar_sync(1, 256);
}

// kWhole: H~ is formed here, too.
template <bool kWhole>
__global__ void __launch_bounds__(kSmallThreads, 2)
    multi_small_kernel(const __grid_constant__ SmallMaps maps, const __grid_constant__ SmallParams p) {
  const MultiCall& c = p.c;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base_addr - raw_addr);
  float* part = reinterpret_cast<float*>(sbase);                       // [t16][128], over the drained stages
  float* delta = reinterpret_cast<float*>(sbase + p.stages * p.stage_bytes);   // [share][128]
  __shared__ TermShared term;
  __shared__ uint64_t full[kSmallMaxStages], empty[kSmallMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.stages;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * 128;
  const int t0 = static_cast<int>(blockIdx.y) * p.tile;
  const int nt = min(p.tile, c.T - t0);
  const int kb0 = rank * p.kb_per, kb1 = min(p.k_blocks, kb0 + p.kb_per);
  const int r0 = rank * p.share, cnt = max(0, min(nt - r0, p.share));  // this CTA's rows of the tile
  const uint64_t tmo = c.timeout_ns;
  int* status = c.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&acc_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&maps.x);
    if (p.has_w) tma_prefetch_desc(&maps.w);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0 && p.has_w) {
      const uint64_t keep = l2_evict_last(), once = gridDim.y > 1 ? keep : l2_evict_first();
      uint32_t issued = 0, s = 0, parity = 1;         // (a slot's first fill waits for no release)
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&empty[s], parity, abort_flag, tmo, status))) break;
        uint8_t* st = sbase + s * p.stage_bytes;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(p.stage_bytes));
        tma_load_2d_hint(st, &maps.w, kb * kBK, n0, &full[s], once);
        tma_load_2d_hint(st + kATileBytes, &maps.x, kb * kBK, t0, &full[s], keep);
        ++issued;
        if (++s == static_cast<uint32_t>(S)) { s = 0; parity ^= 1; }
      }
      if (!ok)                                        // copies in flight land before the CTA leaves
        for (uint32_t q = 0; q < static_cast<uint32_t>(S); ++q) {
          const uint32_t uses = issued / S + (q < issued % S ? 1u : 0u);
          if (uses == 0) continue;
          const uint64_t b = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(&full[q]), (uses - 1) & 1u) && globaltimer_ns() - b < 100000000ull) {
          }
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && p.has_w) {
      const uint32_t idesc = idesc_bf16_f32(128, static_cast<uint32_t>(p.t16));
      const uint32_t u_w = smem_u32(sbase) >> 4;
      uint32_t s = 0, parity = 0, at = u_w;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&full[s], parity, abort_flag, tmo, status))) break;
        tc_fence_after();
        const uint64_t ad = kDescSw128K | at, bd = kDescSw128K | (at + (kATileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          mma_bf16(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
        mma_commit(&empty[s]);
        at += static_cast<uint32_t>(p.stage_bytes) >> 4;
        if (++s == static_cast<uint32_t>(S)) { s = 0; parity ^= 1; at = u_w; }
      }
      mma_commit(&acc_full);
      if (!ok) {                                      // the MMAs issued finish before tensor memory is freed
        const uint64_t b = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&acc_full), 0) && globaltimer_ns() - b < 100000000ull) {
        }
      }
    }
  } else {
    // ------------------------------------------------ the adapters' term of this CTA's rows
    const int row = (warp & 3) * 32 + lane;           // output column n0 + row = TMEM lane
    const int w8 = warp - 2;                          // 0..7
    const int half = w8 >> 2;
    if (kWhole) whole_term(c, delta, n0, kb0 * kBK, min(c.K, kb1 * kBK), threadIdx.x - 64);
    else adapters_term(c, term, delta, t0 + r0, cnt, n0, threadIdx.x - 64);
    // (whole: the few rows' terms join their products of W here)
    auto own = [&](int t) { return kWhole && t < c.T ? delta[t * 128 + row] : 0.f; };
    // ------------------------------------------------ the accumulator into shared memory
    if (p.has_w) {
      const bool ok = mbar_wait(&acc_full, 0, abort_flag, tmo, status);
      if (__all_sync(0xffffffffu, ok) && kb1 > kb0) {
        tc_fence_after();
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        for (int col = half * 8; col < p.t16; col += 16) {
          uint32_t r8[8];
          tmem_ld8(tmem + lane_base + col, r8);
#pragma unroll
          for (int i = 0; i < 8; ++i) part[(col + i) * 128 + row] = __uint_as_float(r8[i]) + own(col + i);
        }
        tc_fence_before();
      } else {
        for (int col = half; col < p.t16; col += 2) part[col * 128 + row] = own(col);
      }
    } else if (kWhole) {
      for (int t = half; t < c.T; t += 2) part[t * 128 + row] = own(t);
    }
  }
  __syncthreads();
  if (p.splits > 1) cluster_sync();                   // every CTA's partial tile is in place
  if (warp >= 2) {
    // one row of X per warp, 4 output columns per lane: the splits' sums in CTA order
    const int n = n0 + lane * 4;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (c.bias && n < c.N) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        bias[k] = c.bias_f32 ? static_cast<const float*>(c.bias)[n + k] : bf2f(static_cast<const uint16_t*>(c.bias)[n + k]);
    }
    for (int i = warp - 2; i < cnt; i += 8) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (p.has_w || kWhole) {
        const uint32_t at = smem_u32(part + (r0 + i) * 128 + lane * 4);
        if (p.splits > 1) {
          float4 q[8];
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t ra = mapa_shared(at, static_cast<uint32_t>(min(s, p.splits - 1)));
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(q[s].x), "=f"(q[s].y), "=f"(q[s].z), "=f"(q[s].w)
                         : "r"(ra));
          }
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < p.splits) {
              v[0] += q[s].x; v[1] += q[s].y; v[2] += q[s].z; v[3] += q[s].w;
            }
        } else {
          const float4 q = *reinterpret_cast<const float4*>(part + (r0 + i) * 128 + lane * 4);
          v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
        }
      }
      const float4 d = kWhole ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(delta + i * 128 + lane * 4);
      v[0] = (v[0] + bias[0]) + d.x;
      v[1] = (v[1] + bias[1]) + d.y;
      v[2] = (v[2] + bias[2]) + d.z;
      v[3] = (v[3] + bias[3]) + d.w;
      if (n < c.N) {
        const long long o = static_cast<long long>(t0 + r0 + i) * c.ldy + n;
        if (c.y_f32) *reinterpret_cast<float4*>(static_cast<float*>(c.Y) + o) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.Y) + o) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (p.splits > 1) cluster_sync();                   // no CTA leaves while a peer reads its tile
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

int fail(cudaError_t e) {
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

}  // namespace

// Rank rows of the column groups that a tile of 128 columns can meet
static int ranks_of_tile(const MultiCall& c) {
  return c.og % 128 == 0 ? c.R : c.R * std::min(c.G, 127 / c.og + 2);
}

// One or two rows of few ranks: every tile's CTAs read the rows' A again (from L2) and save the first
// kernel.  One row took 7.1 us so and 7.9 with both kernels (1536 -> 3 x 1536, rank 32), 9.7 and 11.2
// (4096 -> 4096, rank 16), 13.5 and 14.3 (5120 -> 5120, rank 64), besides a launch's time on the host; two rows
// of rank 32 8.0 and 8.6, but two of rank 64 11.8 and 10.8 (1536 -> 8960), three of rank 16 14.8 and 13.4.
bool multi_whole(const MultiCall& c) { return c.T <= 2 && c.T * ranks_of_tile(c) <= 64; }

int launch_multi_shrink_small(const MultiCall& c, cudaStream_t stream) {
  if (c.T > kMultiFewRows) return WP_ERR_UNSUPPORTED;
  // a sweep of a CTA's warps covers 1024 of K; up to four CTAs share a longer K while the grid stays
  // within eight CTAs per SM (most of a grid leaves at once where rows share slots)
  const int chunks = (c.G * c.R + 15) / 16;
  int parts = 1;
  while (parts < 4 && parts * 1024 < c.K && 2ll * parts * c.T * chunks <= 8ll * device_sm_count()) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.T * parts, chunks);
  cfg.blockDim = dim3(kShrinkThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, multi_shrink_small_kernel, c, parts);
  return e == cudaSuccess ? WP_OK : fail(e);
}

int launch_multi_small(const MultiCall& c, const void* W, long long ldw, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};              // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(e);
  if (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
    e = cudaFuncSetAttribute(multi_small_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(multi_small_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    if (e != cudaSuccess) return fail(e);
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  SmallParams p{};
  p.c = c;
  p.has_w = W ? 1 : 0;
  const bool whole = multi_whole(c);       // H~ is formed here, too
  p.k_blocks = (c.K + kBK - 1) / kBK;
  const int n_tiles = (c.N + 127) / 128;
  int t_tiles = 0;
  size_t smem = 0;
  for (p.tile = 128;; p.tile /= 2) {
    if (p.tile < 64) return WP_ERR_UNSUPPORTED;
    const int tile = c.T < p.tile ? c.T : p.tile;
    t_tiles = (c.T + p.tile - 1) / p.tile;
    p.t16 = (tile + 15) / 16 * 16;
    p.tmem_cols = p.t16 <= 32 ? 32 : (p.t16 <= 64 ? 64 : 128);
    // K splits (a cluster's CTAs, up to 8, each with at least two K blocks): the count whose busiest
    // SM streams the least of K -- ceil(CTAs / SMs) / splits, the most splits on a tie.  Beyond 256
    // CTAs (of the 304 that 152 SMs hold) the clusters no longer fit side by side: 64 rows of 5120 -> 5120 took 16.5 us with 6
    // splits (240 CTAs), 22.6 with 7 (280) and 18.9 with 3 (120).
    const long long tiles = static_cast<long long>(n_tiles) * t_tiles;
    p.splits = 1;
    double best = 0;
    for (int q = 1; q <= 8 && (q == 1 || (tiles * q <= 256 && p.k_blocks >= 2 * q)); ++q) {
      const double load = static_cast<double>((tiles * q + device_sm_count() - 1) / device_sm_count()) / q;
      if (q == 1 || load <= best) {
        best = load;
        p.splits = q;
      }
    }
    p.kb_per = (p.k_blocks + p.splits - 1) / p.splits;
    p.share = (tile + p.splits - 1) / p.splits;
    p.stage_bytes = kATileBytes + p.t16 * 128;
    const int delta_bytes = whole ? c.T * (512 + ranks_of_tile(c) * 4) : p.share * 128 * 4;
    p.stages = (kSmallSmem - 1024 - delta_bytes) / p.stage_bytes;
    if (p.stages > kSmallMaxStages) p.stages = kSmallMaxStages;
    if (p.stages > p.kb_per) p.stages = p.kb_per;
    // the partial tile [t16][128] fp32 lies over the stages
    while (p.stages * p.stage_bytes < p.t16 * 512) ++p.stages;
    smem = 1024 + static_cast<size_t>(p.stages) * p.stage_bytes + delta_bytes;
    if (smem <= static_cast<size_t>(kSmallSmem) && p.stages <= kSmallMaxStages) break;
  }
  SmallMaps maps{};
  int rc = encode_map_bf16(&maps.x, c.X, c.K, c.T, c.ldx, kBK, p.t16, 128);
  if (rc == WP_OK && W) rc = encode_map_bf16(&maps.w, W, c.K, c.N, ldw, kBK, 128, 128);
  if (rc != WP_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_tiles * p.splits, t_tiles);
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  // alone, the kernel starts after what came before it in the stream
  cfg.attrs = whole ? attr + 1 : attr;
  cfg.numAttrs = whole ? 1 : 2;
  e = whole ? cudaLaunchKernelEx(&cfg, multi_small_kernel<true>, maps, p)
            : cudaLaunchKernelEx(&cfg, multi_small_kernel<false>, maps, p);
  return e == cudaSuccess ? WP_OK : fail(e);
}

}  // namespace wp
