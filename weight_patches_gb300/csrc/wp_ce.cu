// wp_ce.cu -- softmax cross entropy of rows X [T, K] against a vocabulary's weight W [V, K], and its
// gradients, without keeping the logits z = s X W^T:
//
//   lse[t] = log sum_v exp z[t, v],   loss[t] = lse[t] - z[t, y_t]
//   G[t, v] = dloss[t] s (exp(z[t, v] - lse[t]) - [v = y_t]),   dX = G W,   dW = G^T X
//
// Everything is a matrix product, so everything runs on one tcgen05 kernel of CTA pairs (256 x 256
// tiles, operands by TMA through six stages, two accumulators in tensor memory) in four forms:
//
//   kCeLoss   z tile by tile; the epilogue keeps each row's running maximum and sum of exponentials
//             over the tiles of its unit and leaves one (maximum, sum) per row and unit, which
//             ce_join_kernel puts together.  No logit reaches memory.
//   kCeGrad   z again, over a piece of the vocabulary; the epilogue turns it into G's rows, each
//             divided by its target's entry, rounded once to bf16 (the operand type of the two products
//             below, which sum in fp32; see ce_pack_kernel).
//   kCeDx     G W over the piece: fp32 planes [split][row][K], added up piece by piece (a bulk
//             reduction: one addition per element and piece, in the stream's order).
//   kCeDw     G^T X: the piece's rows of dW, each written once.
//
// Rows that do not count (y_t outside the vocabulary) are left out: ce_pack_kernel copies the rows that
// do next to each other first, and the products run over those alone, so an ignored row costs nothing and
// nothing in it (not even NaN) reaches a gradient.  Their number stays on the device.  (The loss of up to 256 rows has a
// kernel of its own, ce_few_kernel, which computes them all.)
#include <algorithm>
#include <cmath>

#include <cuda.h>
#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

enum { kCeLoss = 0, kCeGrad = 1, kCeDx = 2, kCeDw = 3 };

constexpr int kCeThreads = 384;              // warp 0 TMA, warp 1 MMA, warps 2 and 3 idle, warps 4..11 epilogue
constexpr int kCeEpi0 = 4;
constexpr int kCeEpiWarps = 8;               // two warpgroups, each half of a tile's columns
constexpr int kCeStages = 6;
constexpr int kCeStageBytes = 2 * kATileBytes;
constexpr int kCeSmem = 1024 + kCeStages * kCeStageBytes + 2 * kStgBytes + 256;

// The tensor core adds the 16 products of an MMA step to its accumulator cut towards zero, which
// over the steps of a long K leaves every logit a little small (by about 2^-25 of it a step); a loss has to be good
// to fp32.  So a tile's K is taken in chunks of this many 64-wide blocks, which the epilogue adds up
// in registers (rounding to nearest) while the next chunk runs in the other accumulator.  Off 64 bits (512 rows of 4096,
// 32000 columns; in float32 products of another order 6.2e-7), and the time (6144 rows that count, 4096 x 131072): 4
// blocks 1.5e-7, 4.19 ms; 8 blocks 2.8e-7, 3.90 ms; 16 blocks 6.2e-7, 3.76 ms; in one piece 3.74 ms.
//
// The backward's logits and its products, dX's over the vocabulary and dW's over the rows, take 64 blocks at a time, cut 256 times,
// for G is rounded to bf16 anyway.  (In one piece the error grows with the length: an entry of G of rows of 2^20 was 18 %
// off, dW of 2^20 rows 3.7e-3.)  A sum's chunks are of equal length: a last one of two blocks would wait for the accumulator.
// Time, 16 blocks, 64, in one piece: 2048 x 2048 x 65536 with dW 925, 898, 886 us; 4096 x 4096 x 131072, dX, 4210, 3990, 3987 us;
// 64 rows with dW 565, 566, 626 us (the accumulator is free again before its sums are stored).
constexpr int kCeChunk = 16, kCeSumChunk = 64;

// Rows that count up to which Xs (see ce_pack_kernel) has two parts: dW's products twice, 8 blocks of 64 rows more beside
// the K / 64 of every tile of G and dX.  Beyond, its one part rounds each term of dW a second time.
constexpr int kCeTwoParts = 512;

struct CeParams {
  const int* count;            // rows that count: n
  int mt, nt;                  // kCeDw: row tiles (of the vocabulary piece); column tiles
  int kb;                      // 64-wide blocks of the contraction (kCeDw: of n rows, from count)
  int kb0;                     // kCeDx: those of the first piece
  int pairs;                   // CTA pairs of a full device
  int gm;                      // kCeLoss, kCeGrad: row blocks swept together
  int run;                     // kCeLoss: column tiles per unit
  int splits;                  // kCeDx: at most so many splits of the contraction
  int plane;                   // kCeDx: rows of a plane
  int V;                       // vocabulary
  int v0;                      // first vocabulary row of the piece
  int K;
  int add;                     // kCeDx: add to what the planes hold
  int out_f32;                 // kCeDw
  float c2;                    // logit scale * log2 e
  const int* target;           // compact rows: y, and for kCeGrad the exponent's offset and the target's entry
  const float* lse2;
  const float* tval;
  int lo;                      // kCeDw: X's second part, if the rows are few, follows this many rows on
  float* zt;                   // kCeLoss: log2 e times the target's logit
  float2* part;                // kCeLoss: [2 units of a row][rows]
  int ldpart;
  int* status;
  unsigned long long timeout_ns;
};

struct CeMaps {
  CUtensorMap a, b, y;
};

// One accumulator's worth of work: blocks [kb0, kb1) of the contraction of tile (m, j).
struct CeFill {
  int m, j;                    // row tile, column tile
  int split;
  int kb0, kb1;
  bool first, last;            // the tile's first, last chunk
  bool open, close;            // the unit's first, last fill
};

// dX [n, K]: how many parts the contraction of kb blocks is split into, so that its nt column tiles of each row
// block keep all pairs busy: the count that costs the fewest clocks, the smallest of equals.  A block costs 630 of the
// busiest pair; a further plane's sums, 8 bytes an element, go at about 1100 bytes a clock (3277 x 4096 against pieces of
// 32768: 4.12 ms in one part, 4.60 in four; 1000 x 1536 against 50021: 406 us in one part, 361 in six).  The rows that count are known on
// the device alone, so each kernel that needs the count works it out.
__device__ __forceinline__ int ce_splits(int n, int K, int nt, int kb, int pairs, int most) {
  const int tiles = (n + kPairM - 1) / kPairM * nt;
  const long long plane = static_cast<long long>(n) * K / 138;
  int best = 1;
  long long cost = 0x7fffffffffffffffll;
  for (int s = 1; s <= most && s <= kb; ++s) {
    const int per = (kb + s - 1) / s;
    const long long c = static_cast<long long>((tiles * s + pairs - 1) / pairs) * per * 630 + (s - 1) * plane;
    if (c < cost && (kb + per - 1) / per == s) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// The fills of one CTA pair, in order.
template <int kMode>
struct CeWalk {
  int mb, units, groups_m;     // row tiles, units, row tiles swept together
  int u, step, kblocks;
  int m, j, j1, split;
  int kb0, kb, kb1;            // the tile's blocks, the next of them
  int chunk = kCeChunk;        // at most so many a fill
  int splits, per;             // kCeDx
  __device__ __forceinline__ CeWalk(const CeParams& p, int pair, int npairs) {
    const int n = *p.count;
    step = npairs;
    u = pair - npairs;
    kblocks = p.kb;
    mb = (n + kPairM - 1) / kPairM;
    groups_m = 1;
    if constexpr (kMode == kCeDw) {
      mb = p.mt;
      kblocks = (n + kBK - 1) / kBK * (n <= kCeTwoParts ? 2 : 1);
      units = mb * p.nt;
    } else if constexpr (kMode == kCeDx) {
      // as the first piece's, so that every piece adds to the planes that the first has written
      splits = ce_splits(n, p.K, p.nt, p.kb0, p.pairs, p.splits);
      per = (p.kb0 + splits - 1) / splits;
      splits = (kblocks + per - 1) / per;
      units = mb * p.nt * splits;
    } else {
      // sweeps of about equal height
      const int sweeps = (mb + p.gm - 1) / p.gm;
      groups_m = sweeps > 0 ? (mb + sweeps - 1) / sweeps : 1;
      units = mb * ((p.nt + p.run - 1) / p.run);
    }
    j = j1 = 0;
    kb0 = kb = kb1 = 0;
    m = split = 0;
  }
  __device__ __forceinline__ bool next(const CeParams& p, CeFill& f) {
    bool open = false;
    if (kb >= kb1) {                           // the next tile
      if (kMode != kCeLoss || ++j >= j1) {     // the next unit
        u += step;
        if (u >= units) return false;
        open = true;
        if constexpr (kMode == kCeDx) {
          const int mj = u / splits;
          split = u - mj * splits;
          m = mj / p.nt;
          j = mj - m * p.nt;
        } else if constexpr (kMode == kCeDw) {
          m = u / p.nt;
          j = u - m * p.nt;
        } else {
          const int runs = (p.nt + p.run - 1) / p.run;
          const int g = u / (groups_m * runs);
          const int m0 = g * groups_m;
          const int members = min(groups_m, mb - m0);
          const int w = u - m0 * runs;
          const int r = w / members;
          m = m0 + (w - r * members);
          j = r * p.run;
          j1 = min(p.nt, j + p.run);
        }
      }
      kb0 = kMode == kCeDx ? split * per : 0;
      kb1 = kMode == kCeDx ? min(kblocks, kb0 + per) : kblocks;
      if constexpr (kMode != kCeLoss) {
        const int parts = (kb1 - kb0 + kCeSumChunk - 1) / kCeSumChunk;
        chunk = parts > 1 ? (kb1 - kb0 + parts - 1) / parts : kCeSumChunk;
      }
      kb = kb0;
    }
    f.m = m;
    f.j = j;
    f.split = split;
    f.first = kb == kb0;
    f.open = open;
    f.kb0 = kb;
    f.kb1 = kb = min(kb1, kb + chunk);      // (no rows at all, kCeDw: one fill without a block)
    f.last = kb >= kb1;
    f.close = f.last && (kMode != kCeLoss || j + 1 >= j1);
    return true;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Bulk reduction of a shared-memory box into global memory: element-wise fp32 addition.
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, int32_t x, int32_t y, const void* smem_src) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(smem_src))
               : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int32_t x, int32_t y, const void* smem_src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(smem_u32(smem_src))
               : "memory");
}

template <int kMode>
__global__ void __launch_bounds__(kCeThreads, 1)
    ce_kernel(const __grid_constant__ CeMaps maps, const __grid_constant__ CeParams p) {
  constexpr bool kAMn = kMode == kCeDw;                       // A: the outer index runs along the contraction
  constexpr bool kBMn = kMode == kCeDw || kMode == kCeDx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base_addr - raw_addr);
  uint8_t* stg = sbase + kCeStages * kCeStageBytes;           // a staging buffer per epilogue warpgroup
  uint64_t* bars = reinterpret_cast<uint64_t*>(stg + 2 * kStgBytes);
  uint64_t* full = bars;                        // [S]  leader: TMA bytes of both CTAs landed
  uint64_t* empty = bars + kCeStages;           // [S]  both: the pair MMAs consumed the stage
  uint64_t* acc_full = bars + 2 * kCeStages;    // [2]  both: accumulator ready
  uint64_t* acc_empty = acc_full + 2;           // [2]  leader: both CTAs' epilogues drained it
  uint64_t* drain = acc_full + 4;               //      leader: every MMA issued has finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t cta = cluster_ctarank();
  const bool leader = cta == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kCeStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kCeEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int npairs = static_cast<int>(gridDim.x >> 1);
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const uint64_t tmo = p.timeout_ns;
  int* status = p.status;
  // (The waits below acquire at CTA scope: what they order is tensor memory and copies, by their own fences, not
  // another CTA's plain stores.)
  grid_launch_dependents();                     // the next kernel's CTAs get ready as these end
  grid_dependency_wait();                       // the rows, their number and G come from earlier kernels

  // the epilogue holds a row's 128 sums in registers: of the 384 x 168 that the block is launched with, the first
  // warpgroup keeps 56 each and the epilogue's two get 224
  if (warp < kCeEpi0) regs_dec<56>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      const uint32_t full_l0 = mapa_shared(smem_u32(&full[0]), 0);
      CeWalk<kMode> walk(p, pair, npairs);
      CeFill f;
      const int first_part = kMode == kCeDw && *p.count <= kCeTwoParts ? walk.kblocks / 2 : 0x7fffffff;
      while (ok && walk.next(p, f)) {
        const int a0 = f.m * kPairM + static_cast<int>(cta) * kBM;
        const int b0 = f.j * kBN + static_cast<int>(cta) * 128;
        for (int kb = f.kb0; kb < f.kb1; ++kb) {
          if (!(ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag, tmo, status))) break;
          uint8_t* sa = sbase + stage * kCeStageBytes;
          uint8_t* sb = sa + kATileBytes;
          const uint32_t fb = full_l0 + static_cast<uint32_t>(stage) * 8u;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2u * kCeStageBytes);
          if constexpr (kAMn) {
            // G's rows against X's, then once more against X's second part
            const int row = (kb < first_part ? kb : kb - first_part) * kBK;
            tma_load_2d_pair(sa, &maps.a, a0, row, fb);
            tma_load_2d_pair(sa + kATileBytes / 2, &maps.a, a0 + 64, row, fb);
          } else {
            tma_load_2d_pair(sa, &maps.a, kb * kBK, a0, fb);
          }
          if constexpr (kBMn) {
            const int row = kMode == kCeDx       ? kb * kBK + p.v0
                            : kb < first_part ? kb * kBK
                                              : (kb - first_part) * kBK + p.lo;
            tma_load_2d_pair(sb, &maps.b, b0, row, fb);
            tma_load_2d_pair(sb + kATileBytes / 2, &maps.b, b0 + 64, row, fb);
          } else {
            tma_load_2d_pair(sb, &maps.b, kb * kBK, p.v0 + b0, fb);
          }
          ++issued;
          if (++stage == kCeStages) { stage = 0; phase ^= 1; }
        }
      }
      if (!ok && leader) {
        // wait (bounded) for the copies in flight before the CTA exits
        for (uint32_t s = 0; s < kCeStages; ++s) {
          const uint32_t n = issued / kCeStages + (s < issued % kCeStages ? 1u : 0u);
          if (n == 0) continue;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait_cluster(smem_u32(&full[s]), (n - 1) & 1u) && globaltimer_ns() - t0 < 100000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = kAMn   ? idesc_bf16_f32_mn(kPairM, kBN)
                                 : kBMn ? idesc_bf16_f32_bmn(kPairM, kBN)
                                        : idesc_bf16_f32(kPairM, kBN);
      constexpr uint64_t abits = kAMn ? kDescSw128MN : kDescSw128K, bbits = kBMn ? kDescSw128MN : kDescSw128K;
      constexpr uint32_t astep = kAMn ? 2048 >> 4 : 2, bstep = kBMn ? 2048 >> 4 : 2;   // per 16 of the contraction
      const uint32_t u_a = smem_u32(sbase) >> 4, u_b = u_a + (kATileBytes >> 4);
      int stage = 0;
      uint32_t phase = 0;
      int count = 0;
      bool ok = true;
      CeWalk<kMode> walk(p, pair, npairs);
      CeFill f;
      while (ok && walk.next(p, f)) {
        if (f.kb1 <= f.kb0) continue;            // no block: the epilogue writes zeros
        const int b = count & 1;
        if (!(ok = mbar_wait(&acc_empty[b], (static_cast<uint32_t>(count >> 1) & 1u) ^ 1u, abort_flag, tmo, status)))
          break;
        tc_fence_after();
        const uint32_t acc = tmem + b * kBN;
        for (int kb = f.kb0; kb < f.kb1; ++kb) {
          if (!(ok = mbar_wait(&full[stage], phase, abort_flag, tmo, status))) break;
          tc_fence_after();
          const uint32_t off = static_cast<uint32_t>(stage) * (kCeStageBytes >> 4);
          const uint64_t ad = abits | (u_a + off), bd = bbits | (u_b + off);
#pragma unroll
          for (uint32_t kk = 0; kk < kBK / 16; ++kk)
            mma_bf16_pair(acc, ad + kk * astep, bd + kk * bstep, idesc, (kb > f.kb0 || kk > 0) ? 1u : 0u);
          mma_commit_pair_mc(&empty[stage], 0x3);
          if (++stage == kCeStages) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        mma_commit_pair_mc(&acc_full[b], 0x3);
        ++count;
      }
      mma_commit_pair_mc(drain, 0x1);            // every MMA finishes before tensor memory is freed
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait_cluster(smem_u32(drain), 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
    }
  } else if (warp >= kCeEpi0) {
    // ------------------------------------------------------------ epilogue
    regs_inc<224>();
    // a thread is a row of the CTA's 128 and one half (eg) of the tile's 256 columns
    const int eg = (warp - kCeEpi0) >> 2;
    const int q = warp & 3;                      // the tensor-memory lanes that this warp may read
    const int row_in_cta = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t bar_main = 1 + 2 * eg, bar_any = 2 + 2 * eg;
    const bool elected = threadIdx.x == (kCeEpi0 + 4 * eg) * 32;
    const uint32_t acc_empty_l0 = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint8_t* buf = stg + eg * kStgBytes;
    const uint32_t rowb = smem_u32(buf) + row_in_cta * 128;
    const int n = *p.count;
    int count = 0;
    bool staged = false;                         // a bulk store may still read the staging buffer
    CeWalk<kMode> walk(p, pair, npairs);
    CeFill f;
    auto wait_acc = [&]() -> bool {
      const bool okw = mbar_wait(&acc_full[count & 1], static_cast<uint32_t>(count >> 1) & 1u, abort_flag, tmo, status);
      if (named_bar_any(!okw, bar_any, 128)) return false;
      tc_fence_after();
      return true;
    };
    auto release_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(acc_empty_l0 + 8u * static_cast<uint32_t>(count & 1));
      ++count;
    };
    auto stg_free = [&]() {
      if (staged && elected) bulk_wait_read_0();
      named_bar_sync(bar_main, 128);
      staged = true;
    };

    float z[128];                                // the row's sums over this half tile
    // adds a chunk to them
    auto gather = [&](const CeFill& f) {
      const uint32_t t0 = tmem + (count & 1) * kBN + lane_base + eg * 128;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32], q[32];
        tmem_ld32x2(t0 + c * 64, r, t0 + c * 64 + 32, q);
        if (f.first) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            z[c * 64 + i] = __uint_as_float(r[i]);
            z[c * 64 + 32 + i] = __uint_as_float(q[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            z[c * 64 + i] += __uint_as_float(r[i]);
            z[c * 64 + 32 + i] += __uint_as_float(q[i]);
          }
        }
      }
      release_acc();
    };
    if constexpr (kMode == kCeLoss) {
      float top = -INFINITY, sum = 0.f;          // running maximum and sum, base 2
      int target = -1;
      while (walk.next(p, f)) {
        const int row = f.m * kPairM + static_cast<int>(cta) * kBM + row_in_cta;
        const bool row_ok = row < n;
        if (f.open) {
          top = -INFINITY;
          sum = 0.f;
          target = row_ok ? p.target[row] : -1;
        }
        // (no barrier joins these warps, so each goes by its own wait)
        const bool okw = mbar_wait(&acc_full[count & 1], static_cast<uint32_t>(count >> 1) & 1u, abort_flag, tmo, status);
        if (!__all_sync(0xffffffffu, okw)) break;
        tc_fence_after();
        gather(f);
        if (!f.last) continue;
        const int col = f.j * kBN + eg * 128;
        const int cols = p.V - col;              // columns of the vocabulary from here
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < 128; ++i) z[i] *= p.c2;
        if (cols < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= cols) z[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 128; ++i) m = fmaxf(m, z[i]);
        const int at = target - col;
        if (__any_sync(0xffffffffu, at >= 0 && at < 128)) {
          float zt = 0.f;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i == at) zt = z[i];
          if (at >= 0 && at < 128) p.zt[row] = zt;
        }
        const float newtop = fmaxf(top, m);
        const float ref = newtop == -INFINITY ? 0.f : newtop;
        float s[4] = {sum * ex2(top - ref), 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i & 3] += ex2(z[i] - ref);
        sum = (s[0] + s[1]) + (s[2] + s[3]);
        top = newtop;
        if (f.close && row_ok) p.part[static_cast<long long>(f.j / p.run * 2 + eg) * p.ldpart + row] = make_float2(top, sum);
      }
    } else if constexpr (kMode == kCeGrad) {
      int target = -1;
      float lse2 = 0.f, tval = 0.f;
      while (walk.next(p, f)) {
        const int row0 = f.m * kPairM + static_cast<int>(cta) * kBM;
        const int row = row0 + row_in_cta;
        const bool row_ok = row < n;
        if (f.first) {
          target = row_ok ? p.target[row] : -1;
          lse2 = row_ok ? p.lse2[row] : 0.f;
          tval = row_ok ? p.tval[row] : 0.f;
        }
        if (!wait_acc()) break;
        gather(f);
        if (!f.last) continue;
        const int pcol = f.j * kBN + eg * 128;   // column within the piece
#pragma unroll
        for (int c = 0; c < 2; ++c) {            // 64 columns to a 128-byte row of the staging buffer
          stg_free();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = p.v0 + pcol + c * 64 + h * 32;
            const int at = target - col, cols = p.V - col;
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = ex2(fmaf(z[c * 64 + h * 32 + i], p.c2, -lse2));
            if (__any_sync(0xffffffffu, at >= 0 && at < 32)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i == at) v[i] = tval;
            }
            if (cols < 32 || !row_ok) {
              // past the vocabulary or the rows: zeros, whatever the exponential made of no data
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i >= cols || !row_ok) v[i] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
              st_shared_v4(rowb + (((h * 4 + u) ^ (row_in_cta & 7)) * 16), pack_bf16x2(v[8 * u], v[8 * u + 1]),
                           pack_bf16x2(v[8 * u + 2], v[8 * u + 3]), pack_bf16x2(v[8 * u + 4], v[8 * u + 5]),
                           pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
          }
          fence_proxy_async_smem();
          named_bar_sync(bar_main, 128);
          if (elected && row0 < n) {
            tma_store_2d(&maps.y, pcol + c * 64, row0, buf);
            bulk_commit();
          }
        }
      }
      if (elected) bulk_wait_all();
    } else {
      // the staging buffer's 128-byte rows to the tile's columns from c on
      auto store = [&](const CeFill& f, int c) {
        fence_proxy_async_smem();
        named_bar_sync(bar_main, 128);
        const int col = f.j * kBN + eg * 128 + c;
        const int row0 = f.m * kPairM + static_cast<int>(cta) * kBM;
        const bool rows = kMode == kCeDx ? row0 < n : p.v0 + row0 < p.V;
        if (elected && rows && col < p.K) {
          const int yrow = kMode == kCeDx ? f.split * p.plane + row0 : p.v0 + row0;
          if (kMode == kCeDx && p.add)
            tma_add_2d(&maps.y, col, yrow, buf);
          else
            tma_store_2d(&maps.y, col, yrow, buf);
          bulk_commit();
        }
      };
      const bool f32 = kMode == kCeDx || p.out_f32;
      while (walk.next(p, f)) {
        if (kMode == kCeDw && n == 0) {          // no row counts, no fill has a block
          const int cw = f32 ? 32 : 64;
#pragma unroll 1
          for (int c = 0; c < 128; c += cw) {
            stg_free();
#pragma unroll
            for (int u = 0; u < 8; ++u) st_shared_v4(rowb + u * 16, 0u, 0u, 0u, 0u);
            store(f, c);
          }
          continue;
        }
        if (!wait_acc()) break;
        gather(f);
        if (!f.last) continue;
        if (f32) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            stg_free();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int i = c * 32 + 4 * u;
              st_shared_v4(rowb + ((u ^ (row_in_cta & 7)) * 16), __float_as_uint(z[i]), __float_as_uint(z[i + 1]),
                           __float_as_uint(z[i + 2]), __float_as_uint(z[i + 3]));
            }
            store(f, c * 32);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            stg_free();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const int i = c * 64 + 8 * u;
              st_shared_v4(rowb + ((u ^ (row_in_cta & 7)) * 16), pack_bf16x2(z[i], z[i + 1]), pack_bf16x2(z[i + 2], z[i + 3]),
                           pack_bf16x2(z[i + 4], z[i + 5]), pack_bf16x2(z[i + 6], z[i + 7]));
            }
            store(f, c * 64);
          }
        }
      }
      if (elected) bulk_wait_all();
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();                               // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------ the rows that count
struct CePack {
  int T, K, V;
  int rows;                    // rows per block
  const void* target; int t64;
  const uint16_t* X; long long ldx;
  uint16_t* Xc;                // [T, K]
  int* count;
  int* from;                   // forward: [T] the row that compact row i was
  int* pos;                    // backward: [T] where row t went, or -1
  int* target_c;
  float* loss; float* lse_out; // forward: zero for the rows that do not count
  const float* lse; const float* dloss;
  // backward
  const uint16_t* W; long long ldw;
  float* lse2_c; float* tval_c; float* rs_c;
  uint16_t* Xs;                // [xs, K]: rs X in one bf16 part, or, of few rows that count, in two
  int lo;                      // rows from the first part to the second
  float scale;
};

__device__ __forceinline__ long long ce_target(const CePack& p, int t) {
  return p.t64 ? static_cast<const long long*>(p.target)[t] : static_cast<const int*>(p.target)[t];
}

// The smallest 1 - p that a row is divided by (below it the row's gradient is lost in its neighbours' anyway).
constexpr float kCeLeast = 0x1p-20f;

// Block b takes p.rows rows.  It counts the rows that count ahead of its own itself (the targets are a
// few bytes a row and stay in L2), so that no block waits for another.
//
// Backward: a row of G is -dloss s (1 - p) at its target and dloss s p_v elsewhere, the p_v adding up to 1 - p.  Held
// in bf16 its largest entry, the target's, would cost dX half a step of each row.  So G is kept divided by
// rs = dloss s (1 - p), which makes that entry -1, exact, and rs goes to the other side: to dX's rows as they are
// finished, in fp32, and for dW into X, Xs = rs X, in two bf16 parts while the rows that count are few and the second
// costs little.
// p comes from the row's product with its target's row of W.
template <bool kBack>
__global__ void __launch_bounds__(256) ce_pack_kernel(const CePack p) {
  grid_launch_dependents();
  __shared__ int red[2][8];
  __shared__ int slot[64];                      // where the rows at hand go, -1: nowhere
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * p.rows;
  int before = 0, total = 0;
#pragma unroll 8
  for (int t = tid; t < p.T; t += 256) {
    const long long y = ce_target(p, t);
    const int v = y >= 0 && y < p.V;
    total += v;
    if (t < r0) before += v;
  }
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    red[0][warp] = before;
    red[1][warp] = total;
  }
  __syncthreads();
  int base = 0, n = 0;
  for (int w = 0; w < 8; ++w) {
    base += red[0][w];
    n += red[1][w];
  }
  const bool two = n <= kCeTwoParts;            // Xs has its second part
  if (blockIdx.x == 0 && tid == 0) *p.count = n;
  const int vecs = p.K >> 3;
  for (int b0 = r0; b0 < min(p.T, r0 + p.rows); b0 += 64) {      // 64 rows at a time
    const int rows = min(64, min(p.T, r0 + p.rows) - b0);
    __syncthreads();
    if (warp == 0) {
      for (int i = lane; i < 64; i += 32) {
        const int t = b0 + i;
        const bool mine = i < rows;
        const long long y = mine ? ce_target(p, t) : -1;
        const bool v = y >= 0 && y < p.V;
        const uint32_t all = __ballot_sync(0xffffffffu, v);
        const int at = v ? base + __popc(all & ((1u << lane) - 1u)) : -1;
        base += __popc(all);
        slot[i] = at;
        if (!mine) continue;
        if (p.pos) p.pos[t] = at;
        if (v) {
          p.target_c[at] = static_cast<int>(y);
          if (p.from) p.from[at] = t;
        } else if (p.loss) {
          p.loss[t] = 0.f;
          if (p.lse_out) p.lse_out[t] = 0.f;
        }
      }
    }
    __syncthreads();
    // a warp a row
    for (int r = warp; r < rows; r += 8) {
      const int at = slot[r], t = b0 + r;
      if (at < 0) continue;
      const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<long long>(t) * p.ldx);
      uint4* xc = reinterpret_cast<uint4*>(p.Xc + static_cast<long long>(at) * p.K);
      if constexpr (!kBack) {
#pragma unroll 8
        for (int c = lane; c < vecs; c += 32) xc[c] = __ldg(x + c);
      } else {
        const uint4* w = reinterpret_cast<const uint4*>(p.W + ce_target(p, t) * p.ldw);
        float z = 0.f;
#pragma unroll 8
        for (int c = lane; c < vecs; c += 32) {
          const uint4 a = __ldg(x + c), b = __ldg(w + c);
          xc[c] = a;
          const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            z = fmaf(__uint_as_float(u[k] << 16), __uint_as_float(v[k] << 16), z);
            z = fmaf(__uint_as_float(u[k] & 0xffff0000u), __uint_as_float(v[k] & 0xffff0000u), z);
          }
        }
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float lse = p.lse[t];
        const float rest = -expm1f(z * p.scale - lse);             // 1 - p
        const float div = rest < kCeLeast ? kCeLeast : rest;       // (a NaN stays one)
        const float rs = p.dloss[t] * p.scale * div;
        if (lane == 0) {
          p.lse2_c[at] = fmaf(lse, 1.4426950408889634f, log2f(div));
          p.tval_c[at] = rest < kCeLeast ? -rest / div : -1.f;
          p.rs_c[at] = rs;
        }
        if (!p.Xs) continue;
        uint4* hi = reinterpret_cast<uint4*>(p.Xs + static_cast<long long>(at) * p.K);
        uint4* lo = reinterpret_cast<uint4*>(p.Xs + (static_cast<long long>(at) + p.lo) * p.K);
        for (int c = lane; c < vecs; c += 32) {
          const uint4 a = __ldg(x + c);
          const uint32_t u[4] = {a.x, a.y, a.z, a.w};
          uint32_t h[4], l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a0 = rs * __uint_as_float(u[k] << 16), a1 = rs * __uint_as_float(u[k] & 0xffff0000u);
            h[k] = pack_bf16x2(a0, a1);
            l[k] = pack_bf16x2(a0 - __uint_as_float(h[k] << 16), a1 - __uint_as_float(h[k] & 0xffff0000u));
          }
          hi[c] = make_uint4(h[0], h[1], h[2], h[3]);
          if (two) lo[c] = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
    }
  }
  if (kBack && p.Xs) {
    // dW's contraction takes rows 64 at a time: zeros from n on to the end of the last 64
    const int end = (n + 63) & ~63;
    for (int r = n + static_cast<int>(blockIdx.x); r < end; r += gridDim.x)
      for (int c = tid; c < vecs; c += 256) {
        reinterpret_cast<uint4*>(p.Xs + static_cast<long long>(r) * p.K)[c] = make_uint4(0, 0, 0, 0);
        if (two) reinterpret_cast<uint4*>(p.Xs + (static_cast<long long>(r) + p.lo) * p.K)[c] = make_uint4(0, 0, 0, 0);
      }
  }
}

// ------------------------------------------------------------------ joining the units' maxima and sums
struct CeJoin {
  const int* count;
  const int* from;
  const float2* part;
  int parts, ldpart;
  const float* zt;
  float* loss;
  float* lse;
};

// 32 rows a block; warp w takes the parts w, w + 32, ... of them, then the warps' results meet in order.
__global__ void __launch_bounds__(1024) ce_join_kernel(const CeJoin p) {
  grid_dependency_wait();
  __shared__ float2 red[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  const int n = *p.count;
  if (blockIdx.x * 32 >= n) return;
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 v) {
    const float nt = fmaxf(top, v.x), ref = nt == -INFINITY ? 0.f : nt;
    sum = sum * ex2(top - ref) + v.y * ex2(v.x - ref);
    top = nt;
  };
  if (row < n) {
    const float2* at = p.part + row;
    int i = warp;
    for (; i + 96 < p.parts; i += 128) {
      float2 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = at[static_cast<long long>(i + 32 * k) * p.ldpart];
#pragma unroll
      for (int k = 0; k < 4; ++k) join(v[k]);
    }
    for (; i < p.parts; i += 32) join(at[static_cast<long long>(i) * p.ldpart]);
  }
  red[warp][lane] = make_float2(top, sum);
  __syncthreads();
  if (warp != 0 || row >= n) return;
  for (int w = 1; w < 32; ++w) join(red[w][lane]);
  const float lse2 = top + log2f(sum);
  const int t = p.from[row];
  constexpr float ln2 = 0.6931471805599453f;
  if (p.loss) p.loss[t] = ((top - p.zt[row]) + log2f(sum)) * ln2;
  if (p.lse) p.lse[t] = lse2 * ln2;
}

// ------------------------------------------------------------------ a few rows
// Up to kCeFewRows rows: W is read once whatever their number, and that is the time there is.  The vocabulary takes the
// MMA's 128 rows and the batch its width (16 to 256), so that the products cost what the rows need; every SM
// streams its own 128-row tiles of W through a ring of all its shared memory, X beside it from L2.  Rows
// that do not count are computed and left out by the join: nothing of a row reaches another's columns.
// (One row of 1536 against 32000: 41 us with the batch on the MMA's 256 rows as in the other form, 24.8 so, of which the
// stream is 15 to 18; 28.7 with W's rows shared out evenly in boxes of 32.  64 rows of 4096 against 131072: 170 us, 6.3 TB/s.)
constexpr int kCeFewRows = 256;

struct CeFewParams {
  int T, V, kb, tiles, stages;
  const void* target; int t64;
  float c2;
  float* zt;
  float2* part;                // [T][4 CTAs]
  int* status;
  unsigned long long timeout_ns;
};

struct CeFewMaps {
  CUtensorMap w, x;
};

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Sums over the warp's lanes of v[0..G-1]; lane l gets that of column l % G.  Each step halves what a lane carries.
template <int G>
__device__ __forceinline__ float lane_sums(float (&v)[G]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o];
      v[i] = (up ? v[i + o] : v[i]) + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float a = v[0];
#pragma unroll
  for (int o = G; o < 32; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// kN: the batch rounded up to the MMA's width.  A thread of the epilogue is a row of the tile (an entry of the
// vocabulary) and half of the batch's columns.
template <int kN>
__global__ void __launch_bounds__(kCeThreads, 1)
    ce_few_kernel(const __grid_constant__ CeFewMaps maps, const __grid_constant__ CeFewParams p) {
  constexpr int C = kN / 2;                                   // columns of a thread
  constexpr int G = C < 32 ? C : 32;                          // taken together
  constexpr uint32_t kXBytes = kN * 128;
  constexpr uint32_t kStage = kATileBytes + kXBytes;
  // K chunks as above, as small as their epilogue fits beside a block's arrival
  constexpr int kChunk = kN <= 16 ? 1 : kN <= 64 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base_addr - raw_addr);
  const int S = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(sbase + S * kStage);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* target = reinterpret_cast<int*>(tmem_slot + 2);        // [kN]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kCeEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kN);
    tmem_relinquish();
  }
  if (warp >= kCeEpi0)
    for (int i = threadIdx.x - kCeEpi0 * 32; i < kN; i += 256) {
      const long long y = i < p.T ? (p.t64 ? static_cast<const long long*>(p.target)[i] : static_cast<const int*>(p.target)[i]) : -1;
      target[i] = y >= 0 && y < p.V ? static_cast<int>(y) : -1;
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const uint64_t tmo = p.timeout_ns;
  int* status = p.status;
  if (kN == 256 && warp < kCeEpi0) regs_dec<56>();
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      const uint64_t keep = l2_evict_last(), once = l2_evict_first();
      for (int tile = blockIdx.x; tile < p.tiles && ok; tile += gridDim.x)
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!(ok = mbar_wait(&empty[stage], phase ^ 1, abort_flag, tmo, status))) break;
          uint8_t* st = sbase + stage * kStage;
          mbar_arrive_expect_tx(&full[stage], kStage);
          tma_load_2d_hint(st, &maps.w, kb * kBK, tile * 128, &full[stage], once);
          tma_load_2d_hint(st + kATileBytes, &maps.x, kb * kBK, 0, &full[stage], keep);
          ++issued;
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
      if (!ok)
        for (uint32_t s = 0; s < static_cast<uint32_t>(S); ++s) {
          const uint32_t n = issued / S + (s < issued % S ? 1u : 0u);
          if (n == 0) continue;
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(&full[s]), (n - 1) & 1u) && globaltimer_ns() - t0 < 100000000ull) {
          }
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, kN);
      const uint32_t u_a = smem_u32(sbase) >> 4;
      int stage = 0, count = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < p.tiles && ok; tile += gridDim.x)
        for (int k0 = 0; k0 < p.kb && ok; k0 += kChunk) {
          const int b = count & 1;
          if (!(ok = mbar_wait(&acc_empty[b], (static_cast<uint32_t>(count >> 1) & 1u) ^ 1u, abort_flag, tmo, status))) break;
          tc_fence_after();
          for (int kb = k0; kb < min(p.kb, k0 + kChunk); ++kb) {
            if (!(ok = mbar_wait(&full[stage], phase, abort_flag, tmo, status))) break;
            tc_fence_after();
            const uint32_t at = u_a + static_cast<uint32_t>(stage) * (kStage >> 4);
            const uint64_t ad = kDescSw128K | at, bd = kDescSw128K | (at + (kATileBytes >> 4));
#pragma unroll
            for (uint32_t kk = 0; kk < kBK / 16; ++kk)
              mma_bf16(tmem + b * kN, ad + 2 * kk, bd + 2 * kk, idesc, (kb > k0 || kk > 0) ? 1u : 0u);
            mma_commit(&empty[stage]);
            if (++stage == S) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          mma_commit(&acc_full[b]);
          ++count;
        }
      mma_commit(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(drain), 0) && globaltimer_ns() - t0 < 100000000ull) {
      }
    }
  } else if (warp >= kCeEpi0) {
    if (kN == 256) regs_inc<224>();
    const int eg = (warp - kCeEpi0) >> 2, q = warp & 3;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    float z[C];
    float top[C / G], sum[C / G];              // of column lane % G of each group, over this warp's tiles
#pragma unroll
    for (int i = 0; i < C / G; ++i) {
      top[i] = -INFINITY;
      sum[i] = 0.f;
    }
    int count = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < p.tiles && ok; tile += gridDim.x) {
      for (int k0 = 0; k0 < p.kb; k0 += kChunk) {
        const bool okw = mbar_wait(&acc_full[count & 1], static_cast<uint32_t>(count >> 1) & 1u, abort_flag, tmo, status);
        if (!(ok = __all_sync(0xffffffffu, okw))) break;
        tc_fence_after();
        const uint32_t t0 = tmem + (count & 1) * kN + lane_base + eg * C;
        auto put = [&](int at, uint32_t r) { z[at] = k0 == 0 ? __uint_as_float(r) : z[at] + __uint_as_float(r); };
        if constexpr (C == 8) {
          uint32_t r[8];
          tmem_ld8(t0, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) put(i, r[i]);
        } else if constexpr (C == 16) {
          uint32_t a[8], b[8];
          tmem_ld8(t0, a);
          tmem_ld8(t0 + 8, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            put(i, a[i]);
            put(8 + i, b[i]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < C / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(t0 + c * 32, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) put(c * 32 + i, r[i]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[count & 1]);
        ++count;
      }
      if (!ok) break;
      const int v = tile * 128 + q * 32 + lane;
      const bool real = v < p.V;
#pragma unroll
      for (int g = 0; g < C / G; ++g) {
        float mine = -INFINITY, e[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const float x = real ? z[g * G + i] * p.c2 : -INFINITY;
          const int col = eg * C + g * G + i;
          if (real && target[col] == v) p.zt[col] = x;
          const float m = warp_max(x);
          e[i] = ex2(x - (m == -INFINITY ? 0.f : m));
          if ((lane & (G - 1)) == i) mine = m;
        }
        const float s = lane_sums<G>(e);
        const float nt = fmaxf(top[g], mine), ref = nt == -INFINITY ? 0.f : nt;
        sum[g] = sum[g] * ex2(top[g] - ref) + s * ex2(mine - ref);
        top[g] = nt;
      }
    }
    if (ok && lane < G)
#pragma unroll
      for (int g = 0; g < C / G; ++g) {
        const int col = eg * C + g * G + lane;
        if (col < p.T) p.part[static_cast<long long>(col) * (4 * gridDim.x) + blockIdx.x * 4 + q] = make_float2(top[g], sum[g]);
      }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * kN);
  }
}

struct CeFewJoin {
  const void* target; int t64;
  int V, parts;
  const float2* part;
  const float* zt;
  float* loss;
  float* lse;
};

// A block a row; every thread's parts, then the threads' results in order.
__global__ void __launch_bounds__(256) ce_few_join_kernel(const CeFewJoin p) {
  __shared__ float2 red[8];
  const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long y = p.t64 ? static_cast<const long long*>(p.target)[row] : static_cast<const int*>(p.target)[row];
  const bool counts = y >= 0 && y < p.V;
  grid_dependency_wait();
  float top = -INFINITY, sum = 0.f;
  auto join = [&](float2 v) {
    const float nt = fmaxf(top, v.x), ref = nt == -INFINITY ? 0.f : nt;
    sum = sum * ex2(top - ref) + v.y * ex2(v.x - ref);
    top = nt;
  };
  const float2* at = p.part + static_cast<long long>(row) * p.parts;
#pragma unroll 4
  for (int i = threadIdx.x; i < p.parts; i += 256) join(at[i]);
  for (int o = 16; o > 0; o >>= 1) {
    // both sides join lower lane first, so that they agree to the bit
    const float2 other = make_float2(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, sum, o));
    const float2 own = make_float2(top, sum);
    const float2 a = lane & o ? other : own, b = lane & o ? own : other;
    top = a.x;
    sum = a.y;
    join(b);
  }
  if (lane == 0) red[warp] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x != 0) return;
  top = red[0].x;
  sum = red[0].y;
  for (int w = 1; w < 8; ++w) join(red[w]);
  constexpr float ln2 = 0.6931471805599453f;
  const float l2 = log2f(sum);
  if (p.loss) p.loss[row] = counts ? ((top - p.zt[row]) + l2) * ln2 : 0.f;
  if (p.lse) p.lse[row] = counts ? (top + l2) * ln2 : 0.f;
}

// ------------------------------------------------------------------ dX from its planes
struct CeFinish {
  int T, K;
  const int* count;
  int nt, kb0, pairs, splits;  // as kCeDx has them
  long long plane;             // elements of a plane
  const float* planes;
  const float* rs;
  const int* pos;
  void* dx; long long ld; int f32;
};

// A block a row at a time.
__global__ void __launch_bounds__(256) ce_finish_kernel(const CeFinish p) {
  __shared__ int count;
  grid_dependency_wait();
  if (threadIdx.x == 0) count = ce_splits(*p.count, p.K, p.nt, p.kb0, p.pairs, p.splits);
  __syncthreads();
  const int splits = count;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    const int at = p.pos[t];
    const float rs = at >= 0 ? p.rs[at] : 0.f;
    for (int c = threadIdx.x * 8; c < p.K; c += 2048) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (at >= 0) {
        const float* src = p.planes + static_cast<long long>(at) * p.K + c;
        for (int s = 0; s < splits; ++s, src += p.plane) {
          const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
          v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
          v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= rs;
      }
      if (p.f32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.dx) + t * p.ld + c);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        st_global_v4(static_cast<uint16_t*>(p.dx) + t * p.ld + c, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      }
    }
  }
}

// ------------------------------------------------------------------ plans
size_t r256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct CePlan {
  long long T, K, V;
  int kb;                      // 64-wide blocks of K
  int vt;                      // 256-wide tiles of the vocabulary
  int mb;                      // 256-row blocks of T
  int gm;                      // row blocks swept together
  int pairs;                   // CTA pairs of the device
  bool few;                    // forward of a few rows
  int grid;                    // its CTAs
  int run, parts;              // forward: tiles of a unit; parts of a row's sum
  int piece, pieces;           // backward: vocabulary columns at a time (a multiple of 256)
  int splits, gk;              // dX: most splits of a piece's contraction; G's rows (T rounded up to 64)
  int lo;                      // dW: rows from Xs's first part to its second
  long long xs;                // dW: rows of Xs
  long long plane;             // dX: rows of a split's plane
  size_t o_count, o_map, o_target, o_zt, o_lse2, o_tval, o_rs, o_x, o_xs, o_part, o_G, o_planes, total;
};

// G holds at most about this many bytes; a piece is as wide as that allows.  Wider pieces add up dX's
// planes less often and give the products' last rounds less weight; the logits of all rows against the
// whole vocabulary never exist.
constexpr long long kCePieceBytes = 256ll << 20;
// Row blocks whose X is swept over the vocabulary together: their rows stay in L2 while W streams past once.
constexpr long long kCeSweepBytes = 32ll << 20;
constexpr int kCeMaxSplits = 16;

// Units of several tiles of one row block leave fewer parts to join, where there are tiles enough.
int ce_run(long long mb, long long vt, int pairs) {
  return static_cast<int>(std::min(8ll, std::max(1ll, mb * vt / (16ll * pairs))));
}

// The workspace for more rows serves fewer as well: what a smaller batch takes more of (parts of its sums, splits of
// its contraction, a wider piece) is reserved for the batch that takes the most.
CePlan ce_plan(long long T, long long K, long long V, bool back) {
  CePlan q{};
  q.T = T; q.K = K; q.V = V;
  q.kb = static_cast<int>((K + kBK - 1) / kBK);
  q.vt = static_cast<int>((V + kBN - 1) / kBN);
  q.mb = static_cast<int>((T + kPairM - 1) / kPairM);
  q.gm = static_cast<int>(std::max(1ll, kCeSweepBytes / (kPairM * K * 2)));
  q.pairs = std::max(1, device_sm_count() / 2);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += r256(bytes);
    return o;
  };
  if (!back) {
    const long long vt128 = (V + 127) / 128;
    q.grid = static_cast<int>(std::min<long long>(std::max(1, device_sm_count()), vt128));
    const long long few = std::min<long long>(T, kCeFewRows);
    const size_t few_bytes = r256(few * 4) + r256(static_cast<size_t>(few) * q.grid * 4 * 8);
    q.few = T <= kCeFewRows;
    if (q.few) {
      q.parts = 4 * q.grid;
      q.o_zt = take(T * 4);
      q.o_part = take(static_cast<size_t>(T) * q.parts * 8);
      q.total = at;
      return q;
    }
    q.run = ce_run(q.mb, q.vt, q.pairs);
    q.parts = 2 * ((q.vt + q.run - 1) / q.run);
    // the largest of the parts of any batch up to T rows: of each run the most rows that have it
    long long most = static_cast<long long>(q.parts) * T;
    for (int r = 1; r < q.run; ++r) {
      const long long mb = ((r + 1) * 16ll * q.pairs - 1) / q.vt;
      if (mb >= 1) most = std::max(most, 2 * ((q.vt + r - 1) / r) * std::min(T, mb * kPairM));
    }
    q.o_count = take(256);
    q.o_map = take(T * 4);
    q.o_target = take(T * 4);
    q.o_zt = take(T * 4);
    q.o_x = take(T * K * 2);
    q.o_part = take(static_cast<size_t>(most) * 8);
    q.total = std::max(at, few_bytes);
  } else {
    q.o_count = take(256);
    q.o_map = take(T * 4);
    q.o_target = take(T * 4);
    q.run = 1;
    q.gk = static_cast<int>((T + 63) / 64 * 64);
    const long long wide = std::max<long long>(kBN, kCePieceBytes / (2ll * q.gk) / kBN * kBN);
    q.pieces = static_cast<int>((q.vt * static_cast<long long>(kBN) + wide - 1) / wide);
    q.piece = static_cast<int>((q.vt + q.pieces - 1) / q.pieces) * kBN;
    q.pieces = static_cast<int>((q.vt * static_cast<long long>(kBN) + q.piece - 1) / q.piece);
    q.o_lse2 = take(T * 4);
    q.o_tval = take(T * 4);
    q.o_rs = take(T * 4);
    q.o_x = take(T * K * 2);
    q.lo = std::min(q.gk, kCeTwoParts);
    q.xs = std::max(q.gk, 2 * q.lo);           // of all rows one part, of few two
    q.o_xs = take(q.xs * K * 2);
    const long long whole = 2ll * q.gk * q.vt * kBN;
    q.o_G = take(static_cast<size_t>(std::min(whole, std::max(kCePieceBytes, 2ll * q.gk * kBN))));
    // splits: up to 16 units a pair, and 16 in all
    const long long nk = (K + kBN - 1) / kBN;
    q.plane = (T + 127) / 128 * 128;           // a store's box holds 128 rows
    q.splits = static_cast<int>(std::min<long long>(kCeMaxSplits, std::max(1ll, kCeMaxSplits * q.pairs / (q.mb * nk))));
    const long long rows = std::min(kCeMaxSplits * q.plane,
                                    std::max(q.plane, (kCeMaxSplits * static_cast<long long>(q.pairs) + nk - 1) / nk * kPairM));
    q.o_planes = take(static_cast<size_t>(rows) * K * 4);
    q.total = at;
  }
  return q;
}

int map_f32(CUtensorMap* m, void* ptr, long long inner, long long outer, long long ld) {
  return encode_map(m, WP_FP32, ptr, inner, outer, ld, 32, 128, 128);
}
int map_bf16(CUtensorMap* m, const void* ptr, long long inner, long long outer, long long ld, int rows) {
  return encode_map(m, WP_BF16, ptr, inner, outer, ld, 64, rows, 128);
}

// A kernel that waits on the device for the one before it.
template <typename P>
int ce_follow(void (*kernel)(P), const P& p, long long grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

template <int kMode>
int ce_launch(const CeMaps& maps, const CeParams& p, long long units, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(ce_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCeSmem);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return WP_ERR_CUDA;
  }
  // no CTA waits for another but its pair's, so a grid of as many pairs as there are SMs for is safe
  // whether or not all of them run at once
  const int pairs = static_cast<int>(std::min<long long>(std::max(1, device_sm_count() / 2), std::max(1ll, units)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kCeThreads);
  cfg.dynamicSmemBytes = kCeSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, ce_kernel<kMode>, maps, p);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return WP_ERR_CUDA;
  }
  return WP_OK;
}

template <int kN>
int ce_few_launch(const CeFewMaps& maps, const CeFewParams& base, int grid, cudaStream_t stream) {
  CeFewParams p = base;
  constexpr int stage = kATileBytes + kN * 128;
  p.stages = std::min(12, (kSmemLimit - 1024 - 2048) / stage);
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * stage + 2048;
  cudaError_t e = cudaFuncSetAttribute(ce_few_kernel<kN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e == cudaSuccess) {
    ce_few_kernel<kN><<<grid, kCeThreads, smem, stream>>>(maps, p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

int ce_few(const wp_mat* X, const wp_mat* W, const void* target, int t64, double logit_scale, float* loss, float* lse,
           const CePlan& q, char* ws, int* status, cudaStream_t st) {
  const int T = static_cast<int>(q.T);
  const int n = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  CeFewMaps maps{};
  int rc;
  if ((rc = map_bf16(&maps.w, W->data, q.K, q.V, W->ld, 128)) != WP_OK) return rc;
  if ((rc = map_bf16(&maps.x, X->data, q.K, T, X->ld, n)) != WP_OK) return rc;
  CeFewParams p{};
  p.T = T; p.V = static_cast<int>(q.V); p.kb = q.kb;
  p.tiles = static_cast<int>((q.V + 127) / 128);
  p.target = target; p.t64 = t64;
  p.c2 = static_cast<float>(logit_scale * 1.4426950408889634);
  p.zt = reinterpret_cast<float*>(ws + q.o_zt);
  p.part = reinterpret_cast<float2*>(ws + q.o_part);
  p.status = status;
  p.timeout_ns = device_wait_limit_ns();
  rc = n == 16    ? ce_few_launch<16>(maps, p, q.grid, st)
       : n == 32  ? ce_few_launch<32>(maps, p, q.grid, st)
       : n == 64  ? ce_few_launch<64>(maps, p, q.grid, st)
       : n == 128 ? ce_few_launch<128>(maps, p, q.grid, st)
                  : ce_few_launch<256>(maps, p, q.grid, st);
  if (rc != WP_OK) return rc;
  CeFewJoin jn{};
  jn.target = target; jn.t64 = t64;
  jn.V = p.V; jn.parts = q.parts;
  jn.part = p.part; jn.zt = p.zt;
  jn.loss = loss; jn.lse = lse;
  return ce_follow(ce_few_join_kernel, jn, T, 256, st);
}

int launched() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

int ce_zero(const wp_out* o, cudaStream_t st) {
  const size_t esz = o->dtype == WP_FP32 ? 4 : 2;
  const cudaError_t e = cudaMemset2DAsync(o->data, o->ld * esz, 0, o->cols * esz, o->rows, st);
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

// A matrix of one row has no pitch that could be off.
template <typename M>
const M* one_row(const M* m, M* own) {
  if (!m || m->rows != 1) return m;
  *own = *m;
  own->ld = m->cols;
  return own;
}

// X and W of either call
int ce_check(const wp_mat* X, const wp_mat* W) {
  for (const wp_mat* m : {X, W}) {
    if (!m || m->rows < 0 || m->cols <= 0 || (!m->data && m->rows != 0)) return WP_ERR_INVALID;
    if (m->dtype != WP_BF16) return m->dtype == WP_FP32 || m->dtype == WP_NF4 ? WP_ERR_DTYPE : WP_ERR_INVALID;
    if (m->ld < m->cols) return WP_ERR_INVALID;
  }
  if (W->rows == 0) return WP_ERR_INVALID;
  if (X->cols != W->cols) return WP_ERR_SHAPE;
  if (X->cols % 8 || X->ld % 8 || W->ld % 8 || !al16(X->data) || !al16(W->data)) return WP_ERR_ALIGN;
  // row, column and tile numbers are 32-bit, rounded up to tiles of 256
  if (X->rows > 0x3FFFFFFFLL || W->rows > 0x7FFFFE00LL || X->cols > (1 << 24)) return WP_ERR_UNSUPPORTED;
  const long long mb = (X->rows + 255) / 256, vt = (W->rows + 255) / 256, kt = (X->cols + 255) / 256;
  if (mb * vt > 0x7FFFFFFFLL || vt * kt > 0x7FFFFFFFLL || mb * kt * 64 > 0x7FFFFFFFLL) return WP_ERR_UNSUPPORTED;
  return WP_OK;
}

template <bool kBack>
int ce_pack(const CePack& base, const CePlan& q, cudaStream_t st) {
  CePack p = base;
  // about four blocks an SM (a block reads every target, so more blocks for more rows would cost their square)
  const long long want = std::max(1, 4 * device_sm_count());
  p.rows = static_cast<int>(std::max(1ll, (q.T + want - 1) / want));
  ce_pack_kernel<kBack><<<static_cast<unsigned>((q.T + p.rows - 1) / p.rows), 256, 0, st>>>(p);
  return launched();
}

}  // namespace

}  // namespace wp

using namespace wp;

extern "C" {

size_t lora_ce_workspace_size(const wp_mat* X, const wp_mat* W, int32_t backward) {
  wp_mat x, w;
  X = one_row(X, &x);
  W = one_row(W, &w);
  if (ce_check(X, W) != WP_OK || X->rows == 0) return 0;
  return ce_plan(X->rows, X->cols, W->rows, backward != 0).total;
}

int lora_ce_fwd(const wp_mat* X, const wp_mat* W, const void* target, int32_t target_bits, double logit_scale,
                float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  wp_mat x, w;
  X = one_row(X, &x);
  W = one_row(W, &w);
  int rc = ce_check(X, W);
  if (rc != WP_OK) return rc;
  if (target_bits != 32 && target_bits != 64) return WP_ERR_DTYPE;
  if (!std::isfinite(static_cast<float>(logit_scale))) return WP_ERR_INVALID;
  if (X->rows == 0) return WP_OK;
  if (!target || (!loss && !lse)) return WP_ERR_INVALID;
  if (!aligned_element(loss, WP_FP32) || !aligned_element(lse, WP_FP32) ||
      (reinterpret_cast<uintptr_t>(target) & (target_bits / 8 - 1)))
    return WP_ERR_ALIGN;
  const CePlan q = ce_plan(X->rows, X->cols, W->rows, false);
  if (!workspace || workspace_bytes < q.total) return WP_ERR_WORKSPACE;
  if (!al16(workspace)) return WP_ERR_ALIGN;
  int* status = tc_status_ptr();
  if (!status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (q.few) return ce_few(X, W, target, target_bits == 64, logit_scale, loss, lse, q, ws, status, st);
  uint16_t* Xc = reinterpret_cast<uint16_t*>(ws + q.o_x);

  CePack pk{};
  pk.T = static_cast<int>(q.T); pk.K = static_cast<int>(q.K); pk.V = static_cast<int>(q.V);
  pk.target = target; pk.t64 = target_bits == 64;
  pk.X = static_cast<const uint16_t*>(X->data); pk.ldx = X->ld;
  pk.Xc = Xc;
  pk.count = reinterpret_cast<int*>(ws + q.o_count);
  pk.from = reinterpret_cast<int*>(ws + q.o_map);
  pk.target_c = reinterpret_cast<int*>(ws + q.o_target);
  pk.loss = loss; pk.lse_out = lse;

  CeMaps maps{};
  if ((rc = map_bf16(&maps.a, Xc, q.K, q.T, q.K, 128)) != WP_OK) return rc;
  if ((rc = map_bf16(&maps.b, W->data, q.K, q.V, W->ld, 128)) != WP_OK) return rc;
  maps.y = maps.a;
  CeParams p{};
  p.count = pk.count;
  p.nt = q.vt; p.kb = q.kb; p.gm = q.gm; p.run = q.run;
  p.V = pk.V; p.K = pk.K;
  p.c2 = static_cast<float>(logit_scale * 1.4426950408889634);
  p.target = pk.target_c;
  p.zt = reinterpret_cast<float*>(ws + q.o_zt);
  p.part = reinterpret_cast<float2*>(ws + q.o_part);
  p.ldpart = pk.T;
  p.status = status;
  p.timeout_ns = device_wait_limit_ns();

  if (loss == nullptr) {
    // the rows that do not count are marked through loss; lse alone takes its place
    pk.loss = lse;
    pk.lse_out = nullptr;
  }
  if ((rc = ce_pack<false>(pk, q, st)) != WP_OK) return rc;
  if ((rc = ce_launch<kCeLoss>(maps, p, static_cast<long long>(q.mb) * ((q.vt + q.run - 1) / q.run), st)) != WP_OK)
    return rc;
  CeJoin jn{};
  jn.count = pk.count; jn.from = pk.from;
  jn.part = p.part; jn.parts = q.parts; jn.ldpart = pk.T;
  jn.zt = p.zt; jn.loss = loss; jn.lse = lse;
  return ce_follow(ce_join_kernel, jn, (q.T + 31) / 32, 1024, st);
}

int lora_ce_bwd(const wp_mat* X, const wp_mat* W, const void* target, int32_t target_bits, const float* lse,
                const float* dloss, double logit_scale, const wp_out* dX, const wp_out* dW, void* workspace,
                size_t workspace_bytes, void* stream) {
  wp_mat x, w;
  wp_out dx1, dw1;
  X = one_row(X, &x);
  W = one_row(W, &w);
  dX = one_row(dX, &dx1);
  dW = one_row(dW, &dw1);
  int rc = ce_check(X, W);
  if (rc != WP_OK) return rc;
  if (target_bits != 32 && target_bits != 64) return WP_ERR_DTYPE;
  if (!std::isfinite(static_cast<float>(logit_scale))) return WP_ERR_INVALID;
  const wp_out* outs[2] = {dX, dW};
  const wp_mat* like[2] = {X, W};
  for (int i = 0; i < 2; ++i) {
    const wp_out* o = outs[i];
    if (!o) continue;
    if (o->rows < 0 || o->cols <= 0 || o->ld < o->cols || (!o->data && o->rows != 0)) return WP_ERR_INVALID;
    if (o->dtype != WP_BF16 && o->dtype != WP_FP32) return WP_ERR_DTYPE;
    if (o->rows != like[i]->rows || o->cols != like[i]->cols) return WP_ERR_SHAPE;
    if (o->ld % (o->dtype == WP_FP32 ? 4 : 8) || !al16(o->data)) return WP_ERR_ALIGN;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (X->rows == 0) return dW ? ce_zero(dW, st) : WP_OK;
  if (!dX && !dW) return WP_OK;
  if (!target || !lse || !dloss) return WP_ERR_INVALID;
  if (!aligned_element(lse, WP_FP32) || !aligned_element(dloss, WP_FP32) ||
      (reinterpret_cast<uintptr_t>(target) & (target_bits / 8 - 1)))
    return WP_ERR_ALIGN;
  const CePlan q = ce_plan(X->rows, X->cols, W->rows, true);
  if (!workspace || workspace_bytes < q.total) return WP_ERR_WORKSPACE;
  if (!al16(workspace)) return WP_ERR_ALIGN;
  int* status = tc_status_ptr();
  if (!status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  char* ws = static_cast<char*>(workspace);
  uint16_t* Xc = reinterpret_cast<uint16_t*>(ws + q.o_x);
  uint16_t* G = reinterpret_cast<uint16_t*>(ws + q.o_G);
  float* planes = reinterpret_cast<float*>(ws + q.o_planes);

  CePack pk{};
  pk.T = static_cast<int>(q.T); pk.K = static_cast<int>(q.K); pk.V = static_cast<int>(q.V);
  pk.target = target; pk.t64 = target_bits == 64;
  pk.X = static_cast<const uint16_t*>(X->data); pk.ldx = X->ld;
  pk.Xc = Xc;
  pk.count = reinterpret_cast<int*>(ws + q.o_count);
  pk.pos = reinterpret_cast<int*>(ws + q.o_map);
  pk.target_c = reinterpret_cast<int*>(ws + q.o_target);
  pk.lse = lse; pk.dloss = dloss;
  pk.W = static_cast<const uint16_t*>(W->data); pk.ldw = W->ld;
  pk.lse2_c = reinterpret_cast<float*>(ws + q.o_lse2);
  pk.tval_c = reinterpret_cast<float*>(ws + q.o_tval);
  pk.rs_c = reinterpret_cast<float*>(ws + q.o_rs);
  pk.Xs = dW ? reinterpret_cast<uint16_t*>(ws + q.o_xs) : nullptr;
  pk.lo = q.lo;
  pk.scale = static_cast<float>(logit_scale);

  CeMaps grad{}, dx{}, dw{};
  if ((rc = map_bf16(&grad.a, Xc, q.K, q.T, q.K, 128)) != WP_OK) return rc;
  if ((rc = map_bf16(&grad.b, W->data, q.K, q.V, W->ld, 128)) != WP_OK) return rc;
  if ((rc = map_bf16(&grad.y, G, q.piece, q.gk, q.piece, 128)) != WP_OK) return rc;
  if (dX) {
    dx.a = grad.y;
    if ((rc = map_bf16(&dx.b, W->data, q.K, q.V, W->ld, 64)) != WP_OK) return rc;
    if ((rc = map_f32(&dx.y, planes, q.K, q.splits * q.plane, q.K)) != WP_OK) return rc;
  }
  if (dW) {
    if ((rc = map_bf16(&dw.a, G, q.piece, q.gk, q.piece, 64)) != WP_OK) return rc;
    if ((rc = map_bf16(&dw.b, pk.Xs, q.K, q.xs, q.K, 64)) != WP_OK) return rc;
    rc = dW->dtype == WP_FP32 ? map_f32(&dw.y, dW->data, q.K, q.V, dW->ld) : map_bf16(&dw.y, dW->data, q.K, q.V, dW->ld, 128);
    if (rc != WP_OK) return rc;
  }
  CeParams p{};
  p.count = pk.count;
  p.gm = q.gm; p.run = 1;
  p.splits = q.splits; p.plane = static_cast<int>(q.plane);
  p.kb0 = static_cast<int>((std::min<long long>(q.piece, q.V) + kBK - 1) / kBK);
  p.pairs = q.pairs;
  p.V = pk.V; p.K = pk.K;
  p.c2 = static_cast<float>(logit_scale * 1.4426950408889634);
  p.out_f32 = dW && dW->dtype == WP_FP32;
  p.target = pk.target_c; p.lse2 = pk.lse2_c; p.tval = pk.tval_c; p.lo = pk.lo;
  p.status = status;
  p.timeout_ns = device_wait_limit_ns();
  const int nk = static_cast<int>((q.K + kBN - 1) / kBN);

  if ((rc = ce_pack<true>(pk, q, st)) != WP_OK) return rc;
  for (int i = 0; i < q.pieces; ++i) {
    const long long v0 = static_cast<long long>(i) * q.piece;
    const long long cols = std::min<long long>(q.piece, q.V - v0);
    const int vt = static_cast<int>((cols + kBN - 1) / kBN);
    p.v0 = static_cast<int>(v0);
    p.nt = vt; p.kb = q.kb;
    if ((rc = ce_launch<kCeGrad>(grad, p, static_cast<long long>(q.mb) * vt, st)) != WP_OK) return rc;
    if (dX) {
      CeParams d = p;
      d.nt = nk;
      d.kb = static_cast<int>((cols + kBK - 1) / kBK);
      // (a last piece with fewer blocks leaves the later splits' planes as the earlier pieces left them)
      d.add = i > 0;
      if ((rc = ce_launch<kCeDx>(dx, d, static_cast<long long>(q.mb) * nk * q.splits, st)) != WP_OK) return rc;
    }
    if (dW) {
      CeParams d = p;
      d.mt = vt; d.nt = nk;
      if ((rc = ce_launch<kCeDw>(dw, d, static_cast<long long>(vt) * nk, st)) != WP_OK) return rc;
    }
  }
  if (dX) {
    CeFinish f{};
    f.T = pk.T; f.K = pk.K;
    f.count = pk.count; f.nt = nk; f.kb0 = p.kb0; f.pairs = q.pairs; f.splits = q.splits;
    f.plane = q.plane * q.K;
    f.planes = planes; f.rs = pk.rs_c; f.pos = pk.pos;
    f.dx = dX->data; f.ld = dX->ld; f.f32 = dX->dtype == WP_FP32;
    return ce_follow(ce_finish_kernel, f, std::min<long long>(q.T, 8ll * device_sm_count()), 256, st);
  }
  return WP_OK;
}

}  // extern "C"
