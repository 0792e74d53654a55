// wp_multi_nf4.cu -- the many-adapter projection of a decode batch over a 4-bit weight.
//
// The codes are the traffic (half a byte a weight) and their decoding is the work.  A byte permute looks
// four codes up in eight bytes: from a pair of 16-entry byte planes of bf16(level * absmax) a weight
// costs two and a half permutes and logic operations, which run at half the issue rate, and
// forming the planes another half when all 64 codes of a block use them.  That is 25 us over 117 million
// weights, so half of the rows go through shared memory's unit instead: a table of the float pairs of
// all 256 code bytes, a packed product with absmax, one conversion for two.  What must not be added is a
// hand-over of decoded tiles between warps: the decoded words go straight into mma.sync fragments.  A
// warp holds 16 weight rows, a lane whole 64-element blocks (q, q + 4, .. with q = lane % 4) of
// rows lane / 4 and lane / 4 + 8, and k is permuted alike on the side of X, so that a lane's four
// consecutive elements are its four of a 16-deep step.  X lies in shared memory once per CTA, placed so
// that the eight lanes of a load's phase hit different banks.  No barrier and no other warp stands
// between a block's load and its sums; two spans of 256 k are on their way while one is worked on.
// K is cut into parts, whose fp32 sums meet in the second kernel with the bias and the adapters' term.
//
// Measured, 28672 x 4096 and 16 slots of rank 16: 16 rows 37 us (this kernel 28, permutes alone 34; the
// codes take 9 from HBM), 1 row 28, 64 rows 79.  With the decoding in warps of its own and
// tcgen05.mma on tiles in shared memory the 16 rows took 54 us, the 64 rows 73; five other layers 12-64 us
// where this takes 9-55.
#include <algorithm>
#include <atomic>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_multi_term.cuh"
#include "wp_nf4.cuh"
#include "wp_ptx.cuh"

namespace wp {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSpan = 256;                // k of a step: four blocks, one a lane of a row
constexpr int kMaxX = 192 * 1024;         // bytes of X a CTA keeps
constexpr int kTable = 256 * 16 * 8;      // bytes of the table of code pairs
constexpr int kSmem = kTable + kMaxX;

struct Nf4Params {
  const uint8_t* codes;                   // [N, K / 2]
  const float* absmax;                    // [N, K / 64]
  const uint16_t* X;
  long long ldx;
  int T, N, K;
  int rows;                               // of X per CTA (blockIdx.y)
  int splits, spans, spans_per;           // parts of K; spans of K in all and a part
  float* part;                            // [splits, T, ldp]
  long long ldp;
  float lv[16];
};

// One block of a row: its 32 code bytes and its scale
struct Block {
  uint4 c[2];
  float am;
};

// Byte planes of the 16 values of a block
struct Planes {
  uint32_t lo[4], hi[4];
  __device__ __forceinline__ Planes(const float (&lv)[16], float am) {
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = pack_bf16x2(lv[2 * k] * am, lv[2 * k + 1] * am);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = prmt(e[2 * j], e[2 * j + 1], 0x6420u);
      hi[j] = prmt(e[2 * j], e[2 * j + 1], 0x7531u);
    }
  }
  // the 8 elements of code word c
  __device__ __forceinline__ void decode(uint32_t c, uint32_t (&o)[4]) const {
    const uint32_t sel = c & 0x77777777u, pick = ((c >> 1) & 0x44444444u) | 0x32103210u;
    lookup4(sel, pick, lo, hi, o[0], o[1]);
    lookup4(sel >> 16, pick >> 16, lo, hi, o[2], o[3]);
  }
};

// The 8 elements of code word c by the table of code pairs (a float pair for each byte, sixteen times
// over, so that the lanes of a half warp read different banks): less work for the permutes' unit, more
// for shared memory's.
__device__ __forceinline__ void decode_by_table(uint32_t c, uint32_t table, float am, uint32_t (&o)[4]) {
  const F2 a = f2(am, am);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t byte = __byte_perm(c, 0, 0x4440 + k);
    F2 v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v.v) : "r"(table + byte * 128));
    float x, y;
    f2_get(f2_mul(v, a), x, y);
    o[k] = pack_bf16x2(x, y);
  }
}

// NT: tiles of 8 rows of X.  kTable2: the second row's blocks go through the table.
template <int NT, bool kTable2>
__global__ void __launch_bounds__(kThreads, 1) multi_nf4_kernel(const __grid_constant__ Nf4Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* xs = smem + (kTable2 ? kTable : 0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  grid_launch_dependents();
  const int part = static_cast<int>(blockIdx.x) % p.splits;
  const int first = part * p.spans_per, ns = min(p.spans_per, p.spans - first);
  const int tiles = (p.N + 15) / 16;
  const int stride_t = static_cast<int>(gridDim.x) / p.splits * kWarps;
  const int tile0 = static_cast<int>(blockIdx.x) / p.splits * kWarps + warp;
  const uint32_t pitch = static_cast<uint32_t>(p.spans_per) * (kSpan * 2);      // bytes of a row of X
  const int blocks = p.K / 64;
  const int t0 = static_cast<int>(blockIdx.y) * p.rows, nt = min(p.rows, p.T - t0);

  // the first blocks of the warp's work, then X, then the walk
  auto fetch = [&](int tile, int s, Block (&b)[2]) {
    const int blk = (first + s) * 4 + q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      b[h].c[0] = b[h].c[1] = make_uint4(0, 0, 0, 0);
      b[h].am = 0.f;
      const int row = min(tile * 16 + g + 8 * h, p.N - 1);
      if (tile < tiles && blk < blocks) {
        const uint4* c = reinterpret_cast<const uint4*>(p.codes + static_cast<long long>(row) * (p.K / 2) + blk * 32);
        b[h].c[0] = __ldg(c);
        b[h].c[1] = __ldg(c + 1);
        b[h].am = __ldg(p.absmax + static_cast<long long>(row) * blocks + blk);
      }
    }
  };
  int tile = tile0, s = 0;                // the step being worked on
  int ft = tile0, fs = 0;                 // the step being fetched
  auto forward = [&](int& t, int& k) {
    if (++k == ns) {
      k = 0;
      t += stride_t;
    }
  };
  Block b[2][2];
  fetch(ft, fs, b[0]);
  forward(ft, fs);
  fetch(ft, fs, b[1]);
  forward(ft, fs);

  if (kTable2)
    for (int i = threadIdx.x; i < 256 * 16; i += kThreads)
      reinterpret_cast<float2*>(smem)[i] = make_float2(p.lv[i >> 8], p.lv[(i >> 4) & 15]);
  const int per_row = p.spans_per * 32;   // 16-byte pieces of a row
  for (int i = threadIdx.x; i < NT * 8 * per_row; i += kThreads) {
    const int r = i / per_row, c = i - r * per_row;
    const long long k = static_cast<long long>(first) * kSpan + c * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < nt && k < p.K) v = __ldg(reinterpret_cast<const uint4*>(p.X + (t0 + r) * p.ldx + k));
    const int place = (c & ~7) | ((c & 7) ^ (((c >> 3) & 3) | (r & 1) << 2));
    *reinterpret_cast<uint4*>(xs + static_cast<size_t>(r) * pitch + place * 16) = v;
  }
  __syncthreads();

  float d[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) d[j][k] = 0.f;
  const uint32_t x0 = smem_u32(xs) + static_cast<uint32_t>(g) * pitch + q * 128;
  const uint32_t turn = static_cast<uint32_t>(q | (g & 1) << 2);

  const uint32_t table = smem_u32(smem) + (lane & 15) * 8;
  auto work = [&](Block (&w)[2]) {
    const Planes p0(p.lv, w[0].am), p1(p.lv, kTable2 ? 0.f : w[1].am);
    const uint32_t c0[8] = {w[0].c[0].x, w[0].c[0].y, w[0].c[0].z, w[0].c[0].w,
                            w[0].c[1].x, w[0].c[1].y, w[0].c[1].z, w[0].c[1].w};
    const uint32_t c1[8] = {w[1].c[0].x, w[1].c[0].y, w[1].c[0].z, w[1].c[0].w,
                            w[1].c[1].x, w[1].c[1].y, w[1].c[1].z, w[1].c[1].w};
    const uint32_t xa = x0 + static_cast<uint32_t>(s) * (kSpan * 2);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint32_t e[4], f[4];
      p0.decode(c0[u], e);
      if (kTable2) decode_by_table(c1[u], table, w[1].am, f);
      else p1.decode(c1[u], f);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint32_t x[4];
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                     : "r"(xa + static_cast<uint32_t>(j) * 8 * pitch + ((u ^ turn) << 4)));
        mma_16816(d[j], e[0], f[0], e[1], f[1], x[0], x[1]);
        mma_16816(d[j], e[2], f[2], e[3], f[3], x[2], x[3]);
      }
    }
    if (s == ns - 1) {
      const int n = tile * 16 + g;
      float* out = p.part + (static_cast<long long>(part) * p.T + t0) * p.ldp + n;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = j * 8 + q * 2 + (k & 1);
          if (t < nt && n + 8 * (k >> 1) < p.N) out[static_cast<long long>(t) * p.ldp + 8 * (k >> 1)] = d[j][k];
          d[j][k] = 0.f;
        }
    }
    forward(tile, s);
  };
  while (tile < tiles) {
    work(b[0]);
    fetch(ft, fs, b[0]);
    forward(ft, fs);
    if (tile >= tiles) break;
    work(b[1]);
    fetch(ft, fs, b[1]);
    forward(ft, fs);
  }
  grid_dependency_wait();                 // this kernel's end stands for the one before it, too
}

// The parts' sums in their order, the bias and the adapters' term of 128 output columns for up to 32
// rows, one rounding.
constexpr int kFinishRows = 32;
__global__ void __launch_bounds__(256) multi_nf4_finish_kernel(const MultiCall c, const float* part, int parts,
                                                              long long ldp) {
  __shared__ TermShared term;
  __shared__ __align__(16) float delta[kFinishRows * 128];
  const int n0 = blockIdx.x * 128, t0 = blockIdx.y * kFinishRows;
  const int cnt = min(kFinishRows, c.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = n0 + lane * 4;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (c.bias && n < c.N) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      bias[k] = c.bias_f32 ? static_cast<const float*>(c.bias)[n + k] : bf2f(static_cast<const uint16_t*>(c.bias)[n + k]);
  }
  adapters_term(c, term, delta, t0, cnt, n0, threadIdx.x);
  __syncthreads();
  if (n >= c.N) return;
  const long long stride = static_cast<long long>(c.T) * ldp;
  for (int i = warp; i < cnt; i += 8) {
    const float* q = part + (t0 + i) * ldp + n;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < parts; k0 += 8) {
      float4 a[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = *reinterpret_cast<const float4*>(q + min(k0 + k, parts - 1) * stride);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k0 + k < parts) {
          v[0] += a[k].x; v[1] += a[k].y; v[2] += a[k].z; v[3] += a[k].w;
        }
    }
    const float4 d = *reinterpret_cast<const float4*>(delta + i * 128 + lane * 4);
    v[0] = (v[0] + bias[0]) + d.x;
    v[1] = (v[1] + bias[1]) + d.y;
    v[2] = (v[2] + bias[2]) + d.z;
    v[3] = (v[3] + bias[3]) + d.w;
    const long long o = (t0 + i) * c.ldy + n;
    if (c.y_f32) *reinterpret_cast<float4*>(static_cast<float*>(c.Y) + o) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(c.Y) + o) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  }
}

template <int NT, bool kTable2>
int launch_nt(const Nf4Params& p, dim3 grid, size_t smem, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !((ready.load(std::memory_order_relaxed) >> dev) & 1u))) {
    e = cudaFuncSetAttribute(multi_nf4_kernel<NT, kTable2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem + (kTable2 ? kTable : 0);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, multi_nf4_kernel<NT, kTable2>, p);
  }
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

// How a call is cut: CTA tiles of up to 64 rows, of equal size; 8-row tiles of the kernel; parts of K.
struct Cut {
  int tiles, rows, nt, parts;
};

// Parts of K: of those that keep X's part in shared memory the one with the least time in nanoseconds: a
// warp's steps (rounds over the row tiles times a part's spans; one took 2.3 us at 16 rows with every warp
// of an SM busy), X's part at 50 bytes, and for each part its sums, written and read at 6 TB/s, and
// the wait for them.
Cut cut_of(int T, int N, int K) {
  Cut c{};
  c.tiles = (T + 63) / 64;
  c.rows = (T + c.tiles - 1) / c.tiles;
  const int eights = (c.rows + 7) / 8;
  c.nt = eights <= 4 ? eights : eights <= 6 ? 6 : 8;
  const int spans = (K + kSpan - 1) / kSpan, tiles = (N + 15) / 16;
  const int most = kMaxX / (c.nt * 8 * kSpan * 2);
  double least = 0;
  for (int per = std::min(most, spans); per >= 1; --per) {
    const int n = (spans + per - 1) / per;
    if ((spans + n - 1) / n != per) continue;        // n parts have fewer spans each
    const int ctas = device_sm_count() / (n * c.tiles);
    if (ctas < 1) break;
    const int round = ctas * kWarps, rounds = (tiles + round - 1) / round;
    const double cost = 2300.0 * rounds * per + c.nt * 8 * per * (kSpan * 2) / 50.0 + n * (400.0 + 8.0 * T * N / 6000.0);
    if (!c.parts || cost < least) {
      c.parts = n;
      least = cost;
    }
  }
  return c;
}

}  // namespace

// Partial sums of the call's rows over the parts of K; 0 parts: K is too long for these kernels.
int multi_nf4_parts(int T, int N, int K) { return cut_of(T, N, K).parts; }

// Rows that are cut alike (as many tiles, as many 8-row tiles of them) differ in a part's price alone, which
// grows with the rows: their parts only become fewer, and the last rows of each count have the most sums.
size_t multi_nf4_most_sums(int T, int N, int K) {
  size_t most = 0;
  for (int t = 1; t <= T;) {
    const Cut c = cut_of(t, N, K);
    int last = std::min(T, c.tiles * c.nt * 8);
    if (cut_of(last, N, K).parts != c.parts) {
      int with = t;                       // has c.parts; `last` has fewer
      while (last - with > 1) {
        const int mid = (with + last) / 2;
        (cut_of(mid, N, K).parts == c.parts ? with : last) = mid;
      }
      last = with;
    }
    most = std::max(most, static_cast<size_t>(c.parts) * last * N);
    t = last + 1;
  }
  return most;
}

int launch_multi_nf4(const MultiCall& c, const void* codes, const float* absmax, float* part, int parts,
                     cudaStream_t stream) {
  Nf4Params p{};
  p.codes = static_cast<const uint8_t*>(codes);
  p.absmax = absmax;
  p.X = c.X; p.ldx = c.ldx;
  p.T = c.T; p.N = c.N; p.K = c.K;
  p.splits = parts;
  p.spans = (c.K + kSpan - 1) / kSpan;
  p.spans_per = (p.spans + parts - 1) / parts;
  p.part = part; p.ldp = c.N;
  nf4_codebook_host(p.lv);
  const Cut cut = cut_of(c.T, c.N, c.K);
  p.rows = cut.rows;
  const int tiles = (c.N + 15) / 16;
  const int ctas = std::max(1, std::min(device_sm_count() / (parts * cut.tiles), (tiles + kWarps - 1) / kWarps));
  const dim3 grid(ctas * parts, cut.tiles);
  const size_t smem = static_cast<size_t>(cut.nt) * 8 * p.spans_per * kSpan * 2;
  int rc;
  switch (cut.nt) {
    case 1: rc = launch_nt<1, true>(p, grid, smem, stream); break;
    case 2: rc = launch_nt<2, true>(p, grid, smem, stream); break;
    case 3: rc = launch_nt<3, true>(p, grid, smem, stream); break;
    case 4: rc = launch_nt<4, true>(p, grid, smem, stream); break;
    case 6: rc = launch_nt<6, false>(p, grid, smem, stream); break;
    default: rc = launch_nt<8, false>(p, grid, smem, stream); break;
  }
  if (rc != WP_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((c.N + 127) / 128, (c.T + kFinishRows - 1) / kFinishRows);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, multi_nf4_finish_kernel, c, static_cast<const float*>(part), parts, p.ldp);
  if (e == cudaSuccess) return WP_OK;
  set_last_cuda_error(e);
  return WP_ERR_CUDA;
}

}  // namespace wp
