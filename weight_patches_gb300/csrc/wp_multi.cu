// wp_multi.cu -- one shared projection for rows that belong to the requests of many adapters.
//
//   Y[t, g] = X[t] W_g^T + bias_g + s_t (X[t] A_{a,g}^T) B_{a,g}^T,   a = slot[t]
//
// (sglang PR, Motivation: the adapter and its scale belong to the request, so a batch meets
// many of them.)  The adapters of a layer lie in a bank, one per slot, and every row names its
// slot on the device.  This file holds the entry point: its checks, its workspace and the choice
// between the forms -- a few rows, where the weights' bytes are the work (wp_multi_small.cu; a 4-bit
// weight in wp_multi_nf4.cu), and many (the blocks' slots and H~ in wp_multi_shrink.cu, then the fused forward of wp_tc_fwd.cu
// with a lane mask per slot).
#include <cmath>

#include <cuda_runtime.h>

#include "wp_internal.h"
#include "wp_ptx.cuh"

namespace wp {

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t r256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

int check(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  if (!X || !bank) return WP_ERR_INVALID;
  if (X->rows < 0 || X->cols <= 0 || X->ld < X->cols) return WP_ERR_INVALID;
  if (X->dtype != WP_BF16 || bank->dtype != WP_BF16) return WP_ERR_DTYPE;
  if (bank->n_slots < 1 || bank->n_groups < 1 || bank->rank < 1 || bank->in <= 0 || bank->out <= 0)
    return WP_ERR_INVALID;
  if (bank->n_groups > kMaxGroups || bank->rank > 256) return WP_ERR_UNSUPPORTED;
  if (bank->in != X->cols || bank->out % bank->n_groups) return WP_ERR_SHAPE;
  if (bank->rank % 8) return WP_ERR_SHAPE;
  if (X->cols % 8 || (bank->out / bank->n_groups) % 8) return WP_ERR_ALIGN;
  // indexes are 32-bit: rows and columns are rounded up to tiles of 512 at most, and the warps of a CTA step
  // through K some thousand at a time, past its end
  if (X->rows > 0x7FFFFFFFll - 512 || X->cols > 0x3FFFFFFFll || bank->out > 0x7FFFFFFFll - 512) return WP_ERR_UNSUPPORTED;
  // the bank's rows are TMA coordinates
  if (bank->n_slots * bank->out > 0x7FFFFFFFll - 512 ||
      static_cast<long long>(bank->n_slots) * bank->n_groups * bank->rank > 0x7FFFFFFFll - 512)
    return WP_ERR_UNSUPPORTED;
  if (W) {
    if (W->dtype != WP_BF16 && W->dtype != WP_NF4) return WP_ERR_DTYPE;
    if (W->rows <= 0 || W->cols <= 0 || W->ld < W->cols) return WP_ERR_INVALID;
    if (W->rows != bank->out || W->cols != bank->in) return WP_ERR_SHAPE;
    if (W->dtype == WP_NF4 && (W->cols % 64 || W->ld != W->cols)) return WP_ERR_SHAPE;
  }
  return WP_OK;
}

// Rows up to which the weight-streaming kernels take a bf16 weight (or none).  At 256 rows they took
// 27-60 us on five layers (1536 -> 4608 and 8960, 4096^2, 5120^2, 8960 -> 1536; 8-16 slots in any order, in runs
// or one) where the masked fused forward took 28-111; at 512 rows of one slot 28-69 against 29-66.
constexpr int kSmallRows = 256;
static_assert(kSmallRows <= kMultiFewRows, "the few-row kernels' lists");
// Rows up to which a 4-bit weight takes the kernels that decode it into fragments: they decode it once per
// 64 rows, the fused forward once per 512.  At 128 rows they took 24-140 us on nine layers (N 1536 to 28672,
// K 1536 to 14336) where the fused forward took 44-176 and in no case 6% more; at 256 rows
// 35-135 against 45-177 on the five with N <= 5120, too few column tiles to fill the fused forward's SMs,
// but 60-287 against 45-142 on the others.
constexpr int kNF4Rows = 128, kNF4RowsNarrow = 256, kNF4Narrow = 5120;
static_assert(kNF4Rows <= kMultiFewRows && kNF4RowsNarrow <= kMultiFewRows, "the few-row kernels' lists");
long long nf4_few_rows(const wp_mat* W) { return W->rows <= kNF4Narrow ? kNF4RowsNarrow : kNF4Rows; }
bool nf4_few(long long T, const wp_mat* W) { return W && W->dtype == WP_NF4 && T <= nf4_few_rows(W); }
bool small_rows(int T, const wp_mat* W) { return T <= kSmallRows && (!W || W->dtype == WP_BF16); }

// H~ [T, G R16] | s [T] (many rows) | entries | their counts | rows with an adapter
// the K splits' partial sums (a 4-bit weight, few rows) come last
struct Layout {
  size_t srow = 0, ent = 0, ent_n = 0, ent_rows = 0, part = 0, total = 0;
  int ent_ld = 0;
  int parts = 0;                          // of K, few rows over a 4-bit weight
};

Layout layout(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  Layout L;
  const size_t T = static_cast<size_t>(X->rows), blocks = (T + 255) / 256;
  const size_t r16 = (bank->rank + 15) / 16 * 16;
  L.srow = r256(T * bank->n_groups * r16 * 2);
  L.total = L.ent = L.srow + r256(T * 4);
  if (!small_rows(static_cast<int>(T < (1u << 30) ? T : (1u << 30)), W)) {
    L.ent_ld = bank->n_slots < 256 ? bank->n_slots : 256;
    L.ent_n = L.ent + r256(blocks * L.ent_ld * sizeof(MultiEntry));
    L.ent_rows = L.ent_n + r256(blocks * 4);
    L.total = L.part = L.ent_rows + r256(blocks * 32);
    if (nf4_few(X->rows, W)) {
      L.parts = multi_nf4_parts(static_cast<int>(T), static_cast<int>(bank->out), static_cast<int>(bank->in));
      L.total += static_cast<size_t>(L.parts) * T * bank->out * 4;
    }
  }
  return L;
}

}  // namespace
}  // namespace wp

using namespace wp;

extern "C" {

size_t lora_multi_workspace_size(const wp_mat* X, const wp_mat* W, const wp_bank* bank) {
  if (check(X, W, bank) != WP_OK || X->rows == 0) return 0;
  const Layout L = layout(X, W, bank);
  if (!W || W->dtype != WP_NF4) return L.total;
  // the partial sums of every call of at most these rows: a workspace for the largest batch serves them all
  // by the same kernels
  const long long few = nf4_few_rows(W) < X->rows ? nf4_few_rows(W) : X->rows;
  return L.part + multi_nf4_most_sums(static_cast<int>(few), static_cast<int>(bank->out), static_cast<int>(bank->in)) * 4;
}

int lora_linear_fwd_multi(const wp_mat* X, const wp_mat* W, const wp_mat* bias, const wp_bank* bank,
                          const int32_t* slot, const float* row_scale, double request_scale,
                          const wp_out* Y, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check(X, W, bank);
  if (rc != WP_OK) return rc;
  if (!Y || Y->rows < 0 || Y->cols <= 0 || Y->ld < Y->cols || (Y->dtype != WP_BF16 && Y->dtype != WP_FP32))
    return WP_ERR_INVALID;
  if (Y->rows != X->rows || Y->cols != bank->out) return WP_ERR_SHAPE;
  const float rs = static_cast<float>(request_scale);
  if (!std::isfinite(rs)) return WP_ERR_INVALID;
  if (bias) {
    if (!bias->data || (bias->dtype != WP_BF16 && bias->dtype != WP_FP32)) return WP_ERR_INVALID;
    if (bias->rows * bias->cols != bank->out || !one_piece(*bias)) return WP_ERR_SHAPE;
  }
  if (X->rows == 0) return WP_OK;
  if (!X->data || !Y->data || !bank->A || !bank->B || !bank->scale || !slot) return WP_ERR_INVALID;
  if (W && (!W->data || (W->dtype == WP_NF4 && !W->absmax))) return WP_ERR_INVALID;
  if (!al16(X->data) || X->ld % 8 || !al16(bank->A) || !al16(bank->B)) return WP_ERR_ALIGN;
  if (W && (!al16(W->data) || W->ld % 8)) return WP_ERR_ALIGN;
  if (!al16(Y->data) || Y->ld % (Y->dtype == WP_BF16 ? 8 : 4)) return WP_ERR_ALIGN;
  if ((bias && !aligned_element(bias->data, bias->dtype)) || (W && !aligned_element(W->absmax, WP_FP32)) ||
      !aligned_element(bank->scale, WP_FP32) || !aligned_element(slot, WP_FP32) || !aligned_element(row_scale, WP_FP32))
    return WP_ERR_ALIGN;
  const Layout L = layout(X, W, bank);
  if (!workspace || workspace_bytes < L.total) return WP_ERR_WORKSPACE;
  if (!al16(workspace)) return WP_ERR_ALIGN;

  char* ws = static_cast<char*>(workspace);
  MultiCall c{};
  c.T = static_cast<int>(X->rows); c.K = static_cast<int>(X->cols); c.N = static_cast<int>(bank->out);
  c.G = bank->n_groups; c.og = c.N / c.G;
  c.R = bank->rank; c.R16 = (c.R + 15) / 16 * 16; c.S = bank->n_slots;
  c.X = static_cast<const uint16_t*>(X->data); c.ldx = X->ld;
  c.A = static_cast<const uint16_t*>(bank->A); c.B = static_cast<const uint16_t*>(bank->B);
  c.scale = bank->scale; c.slot = slot; c.row_scale = row_scale; c.request_scale = rs;
  c.H = reinterpret_cast<uint16_t*>(ws);
  if (bias) {
    c.bias = bias->data;
    c.bias_f32 = bias->dtype == WP_FP32;
  }
  c.Y = Y->data; c.ldy = Y->ld; c.y_f32 = Y->dtype == WP_FP32;
  c.status = tc_status_ptr();
  c.timeout_ns = device_wait_limit_ns();
  if (!c.status) {
    set_last_cuda_error(cudaGetLastError());
    return WP_ERR_CUDA;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (small_rows(c.T, W)) {
    if (!multi_whole(c)) rc = launch_multi_shrink_small(c, st);
    if (rc != WP_OK) return rc;
    return launch_multi_small(c, W ? W->data : nullptr, W ? W->ld : 0, st);
  }
  if (L.parts) {
    rc = launch_multi_shrink_small(c, st);
    if (rc != WP_OK) return rc;
    return launch_multi_nf4(c, W->data, W->absmax, reinterpret_cast<float*>(ws + L.part), L.parts, st);
  }
  c.srow = reinterpret_cast<float*>(ws + L.srow);
  c.ent = reinterpret_cast<MultiEntry*>(ws + L.ent);
  c.ent_n = reinterpret_cast<int*>(ws + L.ent_n);
  c.ent_rows = reinterpret_cast<uint32_t*>(ws + L.ent_rows);
  c.ent_ld = L.ent_ld;
  rc = launch_multi_plan(c, st);
  if (rc == WP_OK) rc = launch_multi_shrink(c, st);
  if (rc == WP_OK) rc = multi_fused(c, W, st);
  return rc;
}

}  // extern "C"
