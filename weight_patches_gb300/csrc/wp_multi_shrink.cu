// wp_multi_shrink.cu -- the many-adapter projection for many rows: which slots each 256-row
// block holds, and H~ = bf16(s X A^T), every row against its own slot.
//
// The rows of a batch come in the scheduler's order: long runs of one slot in prompts, any mixture
// among decoding rows.  Nothing is sorted or copied: a tile of 128 rows of X is multiplied by the
// rank rows of every slot it holds, as many slots side by side as one MMA (N <= 256) and the A ring
// hold -- a small MMA costs its issue, 150 cycles, whatever its width -- and tcgen05.mma's lane mask
// keeps each such group's product in its own rows of the accumulator, where a row's own slot is
// one of the group's column ranges.  A block inside one run costs one product per K step; the
// traffic that no order can avoid is d slots' A, each once per block.
//
// Bound by HBM on X while the blocks hold few slots (96 rank rows: 96 FLOP per byte of X).  Per CTA:
// warp 0 TMA (X and A in rings of their own, since a K step of X serves every group's A), warp 1
// the MMAs, warps 2..5 the output.
// K is split over a cluster when the blocks do not fill the SMs; the partial sums meet in
// distributed shared memory and are added in CTA order.
// The fp32 sums are rounded once to bf16, scaled: the second product takes bf16 operands, and two pieces of
// H~ would double its work, which for a block of many slots is as long as X W^T.  777 rows of
// rank 64 are 1.5 % further from the 64-bit result than with H~ in fp32, Y's own rounding to bf16 the rest
// (lora_linear_fwd rounds alike).
#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

// One CTA per 256-row block.  Distinct slots in the order of their first rows.
__global__ void __launch_bounds__(256) multi_plan_kernel(const MultiCall c) {
  __shared__ int wkey[8][32];
  __shared__ uint32_t wmask[8][32];
  __shared__ int wn[8], wlead[8];
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x * 256 + tid;
  int key = -1;
  if (t < c.T) {
    const int a = c.slot[t];
    float s = 0.f;
    if (a >= 0 && a < c.S) {
      s = c.scale[a];
      if (c.row_scale) s = __fmul_rn(s, c.row_scale[t]);
      s = __fmul_rn(s, c.request_scale);
      if (s != 0.f) key = a;
    }
    c.srow[t] = s;
  }
  // distinct slots of each warp, with their rows
  const uint32_t peers = __match_any_sync(0xffffffffu, key);
  const bool lead = key >= 0 && (peers & ((1u << lane) - 1)) == 0;
  const uint32_t leads = __ballot_sync(0xffffffffu, lead);
  const int at = __popc(leads & ((1u << lane) - 1));
  if (lead) {
    wkey[warp][at] = key;
    wmask[warp][at] = peers;
  }
  const uint32_t rows = __ballot_sync(0xffffffffu, key >= 0);
  if (lane == 0) {
    wn[warp] = __popc(leads);
    c.ent_rows[blockIdx.x * 8 + warp] = rows;
  }
  __syncthreads();
  // a warp's slot leads the block when no earlier warp holds it; its rows in every warp
  bool first = lead;
  uint32_t m[8];
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    m[w] = 0;
    if (lead) {
      const int n = wn[w];
      for (int i = 0; i < n; ++i)
        if (wkey[w][i] == key) m[w] = wmask[w][i];
      if (w < warp && m[w]) first = false;
    }
  }
  const uint32_t firsts = __ballot_sync(0xffffffffu, first);
  if (lane == 0) wlead[warp] = __popc(firsts);
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) base += wlead[w];
    total += wlead[w];
  }
  if (first) {
    MultiEntry& e = c.ent[static_cast<long long>(blockIdx.x) * c.ent_ld + base + __popc(firsts & ((1u << lane) - 1))];
    e.slot = key;
    *reinterpret_cast<uint4*>(e.off) = make_uint4(~m[0], ~m[1], ~m[2], ~m[3]);
    *reinterpret_cast<uint4*>(e.off + 4) = make_uint4(~m[4], ~m[5], ~m[6], ~m[7]);
  }
  if (tid == 0) c.ent_n[blockIdx.x] = total;
}

constexpr int kThreads = 192;
constexpr int kXStages = 3;
constexpr int kMaxAStages = 16;
constexpr int kSmem = 108 * 1024;             // two CTAs per SM, 5 KiB of static arrays each beside it

struct ShrinkMaps {
  CUtensorMap x;               // boxes of 64 K x 128 rows
  CUtensorMap a;               // the bank's A [S G R, K], boxes of 64 K x nc rows
};

struct ShrinkParams {
  MultiCall c;
  int nc;                      // rank rows per CTA (a multiple of 16, at most 128)
  int splits, kb_per, k_blocks;
  int a_area;                  // bytes of the A ring
  int shares;                  // CTAs (blockIdx.z) that share a block's slots
};
constexpr uint32_t kTmemCols = 256;           // two CTAs per SM

__global__ void __launch_bounds__(kThreads, 2)
    multi_shrink_kernel(const __grid_constant__ ShrinkMaps maps, const __grid_constant__ ShrinkParams p) {
  const MultiCall& c = p.c;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base_addr = (raw_addr + 1023u) & ~1023u;
  uint8_t* sx = smem_raw + (base_addr - raw_addr);             // kXStages X tiles
  uint8_t* sa = sx + kXStages * kATileBytes;                   // a_stages A tiles of nc rows
  float* part = reinterpret_cast<float*>(sx);                  // [128][nc + 4], over the drained rings
  __shared__ uint64_t xfull[kXStages], xempty[kXStages], afull[kMaxAStages], aempty[kMaxAStages], acc_full;
  __shared__ int e_slot[128];
  __shared__ __align__(16) uint32_t e_off[128][4];      // read and written 16 bytes at a time
  __shared__ __align__(16) uint32_t g_off[128][4];      // the groups': the lanes that none of its slots owns
  __shared__ __align__(16) uint32_t all_off[4];         // the lanes that no slot of this CTA owns
  __shared__ int e_n;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int blk = static_cast<int>(blockIdx.x) / p.splits;     // 128-row block
  const int t0 = blk * 128;
  const int j0 = static_cast<int>(blockIdx.y) * p.nc;          // first rank row
  const int rows = c.G * c.R;
  const int kb0 = rank * p.kb_per, kb1 = min(p.k_blocks, kb0 + p.kb_per);
  const uint32_t a_bytes = static_cast<uint32_t>(p.nc) * 128;  // one slot's rank rows of a K step
  const uint64_t tmo = c.timeout_ns;
  int* status = c.status;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], 1);
    }
    for (int s = 0; s < kMaxAStages; ++s) {
      mbar_init(&afull[s], 1);
      mbar_init(&aempty[s], 1);
    }
    mbar_init(&acc_full, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&maps.x);
      tma_prefetch_desc(&maps.a);
    }
    // the slots of this half of the 256-row block
    grid_dependency_wait();
    const MultiEntry* ent = c.ent + static_cast<long long>(blk >> 1) * c.ent_ld;
    const int n = c.ent_n[blk >> 1];
    int kept = 0;
    for (int e0 = 0; e0 < n; e0 += 32) {
      uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
      int slot = 0;
      if (e0 + lane < n) {
        m = *reinterpret_cast<const uint4*>(ent[e0 + lane].off + 4 * (blk & 1));
        slot = ent[e0 + lane].slot;
      }
      const bool here = (m.x & m.y & m.z & m.w) != ~0u;
      const uint32_t b = __ballot_sync(0xffffffffu, here);
      if (here) {
        const int at = kept + __popc(b & ((1u << lane) - 1));
        e_slot[at] = slot;
        *reinterpret_cast<uint4*>(e_off[at]) = m;
      }
      kept += __popc(b);
    }
    __syncwarp();
    if (p.shares > 1) {                            // this CTA's share of the slots: whole groups, moved to the front
      const int cap = max(1, min(min(256 / p.nc, p.a_area / (2 * p.nc * 128)), kept));
      const int groups = (kept + cap - 1) / cap, z = static_cast<int>(blockIdx.z);
      const int e0 = z * groups / p.shares * cap, e1 = min(kept, (z + 1) * groups / p.shares * cap);
      kept = max(0, e1 - e0);
      for (int i0 = 0; i0 < kept && e0 > 0; i0 += 32) {
        const int i = min(i0 + lane, kept - 1);
        const int slot = e_slot[e0 + i];
        const uint4 m = *reinterpret_cast<const uint4*>(e_off[e0 + i]);
        __syncwarp();
        e_slot[i] = slot;
        *reinterpret_cast<uint4*>(e_off[i]) = m;
        __syncwarp();
      }
    }
    // the rows of these slots
    uint4 own = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (int e = 0; e < kept; ++e) {
      const uint4 q = *reinterpret_cast<const uint4*>(e_off[e]);
      own.x &= q.x; own.y &= q.y; own.z &= q.z; own.w &= q.w;
    }
    if (lane == 0) {
      e_n = kept;
      *reinterpret_cast<uint4*>(all_off) = own;
    }
    const int gs = max(1, min(min(256 / p.nc, p.a_area / (2 * p.nc * 128)), kept));
    for (int g = lane; g * gs < kept; g += 32) {
      uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
      for (int e = g * gs; e < min(kept, (g + 1) * gs); ++e) {
        const uint4 q = *reinterpret_cast<const uint4*>(e_off[e]);
        m.x &= q.x; m.y &= q.y; m.z &= q.z; m.w &= q.w;
      }
      *reinterpret_cast<uint4*>(g_off[g]) = m;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) grid_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const int ne = e_n;
  // gs slots form a group (one MMA per 16 of K): the most that one MMA's width and half of the A
  // ring hold; SA ring slots of a group each
  int gs = min(min(256 / p.nc, p.a_area / (2 * static_cast<int>(a_bytes))), ne);
  gs = max(gs, 1);
  const int groups = (ne + gs - 1) / gs;
  const uint32_t g_bytes = gs * a_bytes;
  const int SA = min(kMaxAStages, p.a_area / static_cast<int>(g_bytes));

  if (warp == 0) {
    if (lane == 0 && ne > 0) {
      const uint64_t keep = l2_evict_last();
      // ring positions step along (a division by the ring's length would sit on the critical path);
      // xp, ap: the parity of the slot's release that the next fill waits for
      uint32_t xi = 0, ai = 0, xs = 0, as = 0, xp = 1, ap = 1;
      bool ok = true;
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        if (!(ok = mbar_wait(&xempty[xs], xp, abort_flag, tmo, status))) break;
        mbar_arrive_expect_tx(&xfull[xs], kATileBytes);
        tma_load_2d(sx + xs * kATileBytes, &maps.x, kb * kBK, t0, &xfull[xs]);
        ++xi;
        if (++xs == kXStages) { xs = 0; xp ^= 1; }
        for (int e = 0; e < ne; e += gs) {
          if (!(ok = mbar_wait(&aempty[as], ap, abort_flag, tmo, status))) break;
          const int n = min(gs, ne - e);
          mbar_arrive_expect_tx(&afull[as], n * a_bytes);
          for (int i = 0; i < n; ++i)
            tma_load_2d_hint(sa + as * g_bytes + i * a_bytes, &maps.a, kb * kBK, e_slot[e + i] * rows + j0, &afull[as],
                             keep);
          ++ai;
          if (++as == static_cast<uint32_t>(SA)) { as = 0; ap ^= 1; }
        }
      }
      if (!ok) {                                     // copies in flight land before the CTA leaves
        auto settle = [](uint64_t* bar, uint32_t uses) {
          if (uses == 0) return;
          const uint64_t b = globaltimer_ns();
          while (!mbar_try_wait(smem_u32(bar), (uses - 1) & 1u) && globaltimer_ns() - b < 100000000ull) {
          }
        };
        for (uint32_t s = 0; s < kXStages; ++s) settle(&xfull[s], xi / kXStages + (s < xi % kXStages ? 1u : 0u));
        for (uint32_t s = 0; s < static_cast<uint32_t>(SA); ++s) settle(&afull[s], ai / SA + (s < ai % SA ? 1u : 0u));
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc_g = idesc_bf16_f32(128, static_cast<uint32_t>(gs * p.nc));
      const uint32_t idesc_l = idesc_bf16_f32(128, static_cast<uint32_t>((ne - (groups - 1) * gs) * p.nc));
      const uint32_t ux = smem_u32(sx) >> 4, ua = smem_u32(sa) >> 4;
      uint32_t xs = 0, as = 0, xp = 0, ap = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1 && ok && ne > 0; ++kb) {
        if (!(ok = mbar_wait(&xfull[xs], xp, abort_flag, tmo, status))) break;
        const uint64_t ad = kDescSw128K | (ux + xs * (kATileBytes >> 4));
        for (int g = 0; g < groups; ++g) {
          if (!(ok = mbar_wait(&afull[as], ap, abort_flag, tmo, status))) break;
          tc_fence_after();
          const uint64_t bd = kDescSw128K | (ua + as * (g_bytes >> 4));
          const uint4 m = *reinterpret_cast<const uint4*>(g_off[g]);
          const uint32_t off[4] = {m.x, m.y, m.z, m.w};
          const uint32_t idesc = g + 1 < groups ? idesc_g : idesc_l;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma_bf16_lanes(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (kb > kb0 || kk > 0) ? 1u : 0u, off);
          mma_commit(&aempty[as]);
          if (++as == static_cast<uint32_t>(SA)) { as = 0; ap ^= 1; }
        }
        if (!ok) break;
        mma_commit(&xempty[xs]);
        if (++xs == kXStages) { xs = 0; xp ^= 1; }
      }
      mma_commit(&acc_full);
      if (!ok) {
        const uint64_t b = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&acc_full), 0) && globaltimer_ns() - b < 100000000ull) {
        }
      }
    }
  } else {
    // thread = row of the block (its tensor-memory lane); the row's slot is number `mine` of its group
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int t = t0 + row;
    int mine = -1;
    for (int e = 0; e < ne; ++e)
      if (!((e_off[e][row >> 5] >> (row & 31)) & 1u)) mine = e % gs;
    const float s = t < c.T ? c.srow[t] : 0.f;
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full, 0, abort_flag, tmo, status));
    tc_fence_after();
    for (int i = 0; i < gs && ok && ne > 0; ++i) {
      if (__ballot_sync(0xffffffffu, mine == i) == 0) continue;     // (uniform)
      for (int u = 0; u < p.nc / 8; ++u) {
        uint32_t r8[8];
        __syncwarp();
        if (kb1 > kb0) {
          tmem_ld8(tmem + lane_base + i * p.nc + u * 8, r8);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) r8[k] = 0;
        }
        const int j = j0 + u * 8;
        if (mine == i) {
          if (p.splits > 1) {
            float* o = part + row * (p.nc + 4) + u * 8;
            *reinterpret_cast<uint4*>(o) = make_uint4(r8[0], r8[1], r8[2], r8[3]);
            *reinterpret_cast<uint4*>(o + 4) = make_uint4(r8[4], r8[5], r8[6], r8[7]);
          } else if (j < rows) {
            const int g = j / c.R, r = j - g * c.R;
            uint16_t* h = c.H + static_cast<long long>(t) * c.G * c.R16 + g * c.R16 + r;
            auto f = [&](int k) { return __uint_as_float(r8[k]) * s; };
            st_global_v4(h, pack_bf16x2(f(0), f(1)), pack_bf16x2(f(2), f(3)), pack_bf16x2(f(4), f(5)),
                         pack_bf16x2(f(6), f(7)));
            if (c.R != c.R16 && r + 8 == c.R) st_global_v4(h + 8, 0, 0, 0, 0);   // the group's padding columns
          }
        }
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncthreads();
  if (p.splits > 1) {
    cluster_sync();
    // this CTA's share of the rows: 8 rank columns per thread, the splits' sums in CTA order
    const int share = 128 / p.splits, units = p.nc / 8;
    for (int i = threadIdx.x; i < share * units && ne > 0; i += kThreads) {
      const int row = rank * share + i / units, u = i % units;
      const int t = t0 + row, j = j0 + u * 8;
      if (t >= c.T || j >= rows || ((all_off[row >> 5] >> (row & 31)) & 1u)) continue;
      float4 a[8][2];                                  // every split's loads before the first sum
      const uint32_t at = smem_u32(part + row * (p.nc + 4) + u * 8);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t ra = mapa_shared(at, static_cast<uint32_t>(min(q, p.splits - 1)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(a[q][h].x), "=f"(a[q][h].y), "=f"(a[q][h].z), "=f"(a[q][h].w) : "r"(ra + 16 * h));
      }
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < p.splits) {
          v[0] += a[q][0].x; v[1] += a[q][0].y; v[2] += a[q][0].z; v[3] += a[q][0].w;
          v[4] += a[q][1].x; v[5] += a[q][1].y; v[6] += a[q][1].z; v[7] += a[q][1].w;
        }
      const float s = c.srow[t];
      const int g = j / c.R, r = j - g * c.R;
      uint16_t* h = c.H + static_cast<long long>(t) * c.G * c.R16 + g * c.R16 + r;
      st_global_v4(h, pack_bf16x2(v[0] * s, v[1] * s), pack_bf16x2(v[2] * s, v[3] * s),
                   pack_bf16x2(v[4] * s, v[5] * s), pack_bf16x2(v[6] * s, v[7] * s));
      if (c.R != c.R16 && r + 8 == c.R) st_global_v4(h + 8, 0, 0, 0, 0);
    }
    __syncwarp();
    cluster_sync();                                  // no CTA leaves while a peer reads its sums
  }
  // the forward reads H~ by TMA: order these stores for the async proxy
  fence_proxy_async_global();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int fail(cudaError_t e) {
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

}  // namespace

int launch_multi_plan(const MultiCall& c, cudaStream_t stream) {
  multi_plan_kernel<<<(c.T + 255) / 256, 256, 0, stream>>>(c);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? WP_OK : fail(e);
}

int launch_multi_shrink(const MultiCall& c, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};              // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(e);
  if (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u)) {
    e = cudaFuncSetAttribute(multi_shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return fail(e);
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  ShrinkParams p{};
  p.c = c;
  const int rows16 = (c.G * c.R + 15) / 16 * 16;
  const int chunks = (rows16 + 127) / 128;
  p.nc = ((rows16 + chunks - 1) / chunks + 15) / 16 * 16;
  p.k_blocks = (c.K + kBK - 1) / kBK;
  const int blocks = (c.T + 127) / 128;
  p.splits = 1;
  while (p.splits < 8 && 2ll * p.splits * blocks * chunks <= 2ll * device_sm_count() && p.k_blocks >= 4 * p.splits)
    p.splits *= 2;
  p.kb_per = (p.k_blocks + p.splits - 1) / p.splits;
  // Where that leaves SMs idle, the slots a block can hold are shared out as well (X is then read by each
  // share, from L2), up to one and a half CTAs per SM: 777 rows in any order of 12 slots of rank 64 took
  // 19 us with one share, 14 with four, the whole call 56 and 52; 300 rows of 64 such slots 189 and
  // 96.  Rows of one slot, whose other shares find nothing, lose a microsecond.  At two CTAs
  // per SM 1500 rows took 3 to 4 us more than with one share.
  const int a_area = (kSmem - 1024 - kXStages * kATileBytes) / 1024 * 1024;
  const int cap = std::max(1, std::min(256 / p.nc, a_area / (2 * p.nc * 128)));
  const int most = (std::min(c.S, 128) + cap - 1) / cap;
  p.shares = std::max(1, std::min(most, 3 * device_sm_count() / 2 / (blocks * p.splits * chunks)));
  p.a_area = a_area;
  const size_t smem = 1024 + kXStages * kATileBytes + static_cast<size_t>(p.a_area);
  // the partial sums [128][nc + 4] lie over the rings (nc <= 128: 66 KiB of 107)
  ShrinkMaps maps{};
  int rc = encode_map_bf16(&maps.x, c.X, c.K, c.T, c.ldx, kBK, 128, 128);
  if (rc == WP_OK)
    rc = encode_map_bf16(&maps.a, c.A, c.K, static_cast<long long>(c.S) * c.G * c.R, c.K, kBK, p.nc, 128);
  if (rc != WP_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks * p.splits, chunks, p.shares);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, multi_shrink_kernel, maps, p);
  return e == cudaSuccess ? WP_OK : fail(e);
}

}  // namespace wp
