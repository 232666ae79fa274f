// Operators on logit rows around the draft and verify step: shaping of raw
// logits, a teacher's top logits, and the distillation loss against them
// (the entry points declared in include/dspark.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../host_checks.hpp"
#include "distill.hpp"
#include "dspark.h"
#include "shape.hpp"
#include "top.hpp"

namespace dspark {
namespace {

bool temperature_ok(float t) { return t >= 0x1p-100f && t <= 0x1p100f; }

// Output rows beside input rows: the same memory (same type and stride) or
// memory apart.
int check_out(const dspark_rows* in, const void* out, int32_t dtype, int64_t stride) {
  if (stride < in->vocab) return fail(DSPARK_EINVAL, "output stride < vocab");
  const int64_t es = dtype == DSPARK_BF16 ? 2 : 4, ei = in->dtype == DSPARK_BF16 ? 2 : 4;
  if (!aligned16(out) || ((stride * es) & 15) != 0)
    return fail(DSPARK_EALIGN, "output rows must start 16-byte aligned (data and stride * element size)");
  if (in->n_rows == 0) return DSPARK_SUCCESS;
  if (!out) return fail(DSPARK_EINVAL, "NULL output rows");
  if (out == in->data) {
    if (dtype != in->dtype || stride != in->row_stride)
      return fail(DSPARK_EINVAL, "in place needs the input's type and row stride");
    return DSPARK_SUCCESS;
  }
  const char *a = static_cast<const char*>(in->data), *b = static_cast<const char*>(out);
  const char* ae = a + ((in->n_rows - 1) * in->row_stride + in->vocab) * ei;
  const char* be = b + ((in->n_rows - 1) * stride + in->vocab) * es;
  if (a < be && b < ae) return fail(DSPARK_EINVAL, "output rows overlap the input rows");
  return DSPARK_SUCCESS;
}

// ids per slice for `owners` workgroup owners (requests or rows) of V ids
int slice_of(int64_t owners, int64_t V, int64_t most, int64_t want) {
  const int64_t all = (V + kSliceStep - 1) / kSliceStep;                       // groups of a row
  const int64_t n = std::max<int64_t>(1, std::min(all, want / std::max<int64_t>(owners, 1)));  // slices wanted
  const int64_t groups = (all + n - 1) / n;
  return (int)(std::min<int64_t>(groups, most / kSliceStep) * kSliceStep);
}

template <int TI, int TO, int NWV, int G, int DEPTH>
void launch_shape_as(ShapeArgs a, hipStream_t s) {
  constexpr int slice = 64 * NWV * 8 * G;
  a.slices = (a.V + slice - 1) / slice;
  hipLaunchKernelGGL(HIP_KERNEL_NAME(shape_kernel<TI, TO, NWV, G, DEPTH>), row_slice_grid(a.n_requests, a.slices),
                     dim3(64 * NWV), 0, s, a);
}
// What keeps enough loads on their way: two eights of logits per thread and
// two rows ahead (side by side, V = 129,280, 1,024 requests, bf16: 6 rows each 564 us against
// 631 with one eight, three rows ahead and 512 threads, 1 row 196 / 266).
// float32 results need more registers, and with three rows or more the other
// is as fast or faster (float32, 6 rows: 1,139 / 1,104 us, 1 row 204 / 255).
// So is it where the requests leave CUs idle and the history is long, which
// 512 threads scan in half the steps (histories of up to 32,768 tokens, 6
// bf16 rows each: 16 requests 28.0 / 23.5 us, 4 23.7 / 17.6; 64 63.7 / 68.9;
// 24 32.5 / 31.3, where the rounds fit 48 55 / 52 as well and 32 36 / 42).
// bf16 rows with float32 results: 1,024 requests of 6 rows 876 / 868, 64 of 6
// 63.5 / 62.5, but 1,024 of 3 431 / 453, of 2 302 / 345, of 1 217 / 266.
template <int TI, int TO>
void launch_shape(const ShapeArgs& a, hipStream_t s) {
  if (a.V <= 2048) launch_shape_as<TI, TO, 4, 1, 2>(a, s);
  else if ((TO == DSPARK_F32 && a.how.rows_per_request > 2) ||
           (a.how.history && a.how.history_max >= 16384 && a.n_requests * a.V < 1 << 22))
    launch_shape_as<TI, TO, 8, 1, TI == DSPARK_F32 ? 2 : 3>(a, s);
  else launch_shape_as<TI, TO, 4, 2, 2>(a, s);
}

// How dspark_top_logits cuts rows into slices (bytes 0: not at all).  Rows
// longer than kTopSmall always are; shorter ones above 4,096 ids where there
// are 512 or more of them and the sample can place the threshold (k = 64,
// bf16: 1,024 rows of 8,000 ids 16.0 us against 27.6 held whole, of 16,384
// 18.1 / 49.5; 256 rows of 16,384 15.5 / 14.1; 4,096 rows of 4,000 35 / 46).
// The sample's rank leaves four standard deviations above the count expected
// of the top k.
struct TopPlan {
  int slices, cap, rank, most;  // most: candidates that the selection takes
  size_t bytes, part_bytes;
};
TopPlan top_plan(int64_t n, int64_t V, int64_t k_max) {
  TopPlan p{};
  if (V <= kTopSmall && (n < 512 || V <= 4096)) return p;
  const double mu = (double)std::max<int64_t>(std::min(k_max, V), 1) * kTopSample / (double)V;  // < 128 above kTopSmall
  p.rank = (int)std::ceil(mu + 4.0 * std::sqrt(mu) + 4.0);                                      // <= 178 there
  if (V <= kTopSmall && p.rank > 200) return p;
  // logits of the sample above the rank-th of its 256 maxima, and so of a slice and of the row
  const double above = -std::log(1.0 - p.rank / 256.0) * 256.0;
  const double row = above * (double)V / kTopSample;
  // room for more than twice the candidates expected (one row in 1,280 that
  // has to be selected from memory costs more than the selection of all), in
  // workgroups as small as that allows (1,280 bf16 rows, k = 256: 12.3 us in
  // 256 threads of eleven candidates, 15.6 in 512 of eight).  Not so for the
  // longest rows: a sample of 2,048 of 524,288 ids leaves room for 1.9 times as
  // many at k = 1,024, of 1,048,576 ids for 2.0 times (k = 256) to 1.3 (1,024),
  // and 0.3, 1 and 13 % of rows of normal logits pass it.  They are selected
  // from memory (64 rows of 1,048,576 ids, call: bf16 43 us where none is, k =
  // 64, and 790 where some are, k = 256 to 1,024; float32 1,100 to 1,220).
  p.most = row * 2.2 <= 2048 ? 2048 : row * 2.2 <= 2816 ? 2816 : row * 2.2 <= 5632 ? 5632 : 8192;
  p.slices = (int)((V + kTopSlice - 1) / kTopSlice);
  p.cap = (int)std::min<double>(kTopSlice, std::ceil((3.0 * above * kTopSlice / kTopSample + 64.0) / 64.0) * 64.0);
  p.part_bytes = (size_t)n * (size_t)p.slices * sizeof(TopPart);
  p.bytes = (size_t)n * (size_t)p.slices * (size_t)p.cap * 8u + p.part_bytes;
  return p;
}

template <int DT>
void launch_top_slices(const TopSliceArgs& q, const TopPlan& plan, hipStream_t s) {
  hipLaunchKernelGGL(top_slice_kernel<DT>, row_slice_grid(q.a.n, plan.slices), dim3(kSliceBS), 0, s, q);
  const dim3 grid = grid_of(q.a.n);
  if (plan.most == 2048) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_select_kernel<DT, 4, 8>), grid, dim3(256), 0, s, q);
  else if (plan.most == 2816) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_select_kernel<DT, 4, 11>), grid, dim3(256), 0, s, q);
  else if (plan.most == 5632) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_select_kernel<DT, 8, 11>), grid, dim3(512), 0, s, q);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(top_select_kernel<DT, 16, 8>), grid, dim3(1024), 0, s, q);
}

template <int DT>
void launch_top_small(const TopArgs& a, hipStream_t s) {
  const dim3 grid = grid_of(a.n);
  if (a.V <= 2048) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_small_kernel<DT, 4, 1>), grid, dim3(256), 0, s, a);
  else if (a.V <= 4096) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_small_kernel<DT, 8, 1>), grid, dim3(512), 0, s, a);
  else if (a.V <= 8192) hipLaunchKernelGGL(HIP_KERNEL_NAME(top_small_kernel<DT, 16, 1>), grid, dim3(1024), 0, s, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(top_small_kernel<DT, 16, 2>), grid, dim3(1024), 0, s, a);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

int dspark_shape_logits(const dspark_rows* rows, const dspark_shaping* how, void* out, int32_t out_dtype,
                        int64_t out_stride, int32_t* row_status, void* stream) {
  int rc = host_check_rows(rows, "rows NULL");
  if (rc) return rc;
  if (!how) return fail(DSPARK_EINVAL, "NULL shaping");
  if (out_dtype != rows->dtype && out_dtype != DSPARK_F32)
    return fail(DSPARK_EINVAL, "out_dtype must be the rows' type or F32");
  if (how->rows_per_request < 1) return fail(DSPARK_EINVAL, "rows_per_request must be at least 1");
  if (rows->n_rows % how->rows_per_request != 0) return fail(DSPARK_EINVAL, "n_rows is not a multiple of rows_per_request");
  rc = check_out(rows, out, out_dtype, out_stride);
  if (rc) return rc;
  if (how->history && (how->history_max < 0 || how->history_stride < how->history_max || how->history_max > (1 << 30)))
    return fail(DSPARK_EINVAL, "history_max must be in [0, history_stride], at most 2^30");
  if (how->draft && how->draft_stride < how->rows_per_request - 1)
    return fail(DSPARK_EINVAL, "draft_stride < rows_per_request - 1");
  if (how->bias_offset && how->bias_total < 0) return fail(DSPARK_EINVAL, "bias_total < 0");
  if (how->mask && (how->n_masks < 0 || how->mask_stride < (rows->vocab + 31) / 32))
    return fail(DSPARK_EINVAL, "mask_stride is shorter than the vocabulary's bits");
  if (rows->n_rows == 0) return DSPARK_SUCCESS;
  if (!row_status) return fail(DSPARK_EINVAL, "NULL row_status");
  if (how->history && !how->history_len) return fail(DSPARK_EINVAL, "history needs history_len");
  if (how->bias_offset && how->bias_total > 0 && (!how->bias_ids || !how->bias_values))
    return fail(DSPARK_EINVAL, "bias_offset needs bias_ids and bias_values");
  if (how->mask && !how->mask_row && how->n_masks < rows->n_rows)
    return fail(DSPARK_EINVAL, "fewer masks than rows and no mask_row");
  ShapeArgs a;
  a.x = rows->data;
  a.x_stride = rows->row_stride;
  a.out = out;
  a.out_stride = out_stride;
  a.row_status = row_status;
  a.n_requests = rows->n_rows / how->rows_per_request;
  a.V = (int)rows->vocab;
  a.how = *how;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows->dtype == DSPARK_F32) launch_shape<DSPARK_F32, DSPARK_F32>(a, s);
  else if (out_dtype == DSPARK_BF16) launch_shape<DSPARK_BF16, DSPARK_BF16>(a, s);
  else launch_shape<DSPARK_BF16, DSPARK_F32>(a, s);
  return host_check_launch();
}

size_t dspark_top_logits_workspace(int64_t n_rows, int64_t vocab, int32_t k_max) {
  if (n_rows <= 0 || n_rows > (1 << 24) || vocab < 1 || vocab > DSPARK_V_MAX || k_max < 0 || k_max > DSPARK_K_MAX) return 0;
  return top_plan(n_rows, vocab, k_max).bytes;
}

int dspark_top_logits(const dspark_rows* rows, const int32_t* topk, int32_t k_max, float temperature, int32_t* ids,
                      float* logits, int32_t* len, float* lse, int32_t* row_status, void* ws, size_t ws_bytes,
                      void* stream) {
  int rc = host_check_rows(rows, "rows NULL");
  if (rc) return rc;
  if (k_max < 0 || k_max > DSPARK_K_MAX) return fail(DSPARK_EINVAL, "k_max must be in [0, DSPARK_K_MAX]");
  if (!temperature_ok(temperature)) return fail(DSPARK_EINVAL, "temperature must be in [2^-100, 2^100]");
  if (rows->n_rows == 0) return DSPARK_SUCCESS;
  if (!len || !row_status || (k_max > 0 && (!ids || !logits))) return fail(DSPARK_EINVAL, "NULL output");
  const TopPlan plan = top_plan(rows->n_rows, rows->vocab, k_max);
  if (!aligned16(ws)) return fail(DSPARK_EALIGN, "workspace must be 16-byte aligned");
  if (plan.bytes > 0 && (!ws || ws_bytes < plan.bytes))
    return fail(DSPARK_EWORKSPACE, "workspace smaller than dspark_top_logits_workspace()");
  TopSliceArgs q{};
  TopArgs& a = q.a;
  a.n = rows->n_rows;
  a.x = rows->data;
  a.stride = rows->row_stride;
  a.V = (int)rows->vocab;
  a.topk = topk;
  a.k_max = k_max;
  a.inv_t = 1.0 / (double)temperature;
  a.c = (float)(1.4426950408889634 * a.inv_t);
  a.ids = ids;
  a.logits = logits;
  a.len = len;
  a.lse = lse;
  a.row_status = row_status;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (plan.bytes > 0) {
    q.slices = plan.slices;
    q.cap = plan.cap;
    q.rank = plan.rank;
    q.cand = ws;
    q.part = reinterpret_cast<TopPart*>(static_cast<char*>(ws) + plan.bytes - plan.part_bytes);
    if (rows->dtype == DSPARK_F32) launch_top_slices<DSPARK_F32>(q, plan, s);
    else launch_top_slices<DSPARK_BF16>(q, plan, s);
  } else if (rows->dtype == DSPARK_F32) {
    launch_top_small<DSPARK_F32>(a, s);
  } else {
    launch_top_small<DSPARK_BF16>(a, s);
  }
  return host_check_launch();
}

}  // extern "C"

namespace dspark {
namespace {

constexpr int kDistillSliceMost = 32768;
constexpr int kRowMost = 131072;  // ids of a row that one workgroup takes: its set of ids stays below 33 KB of LDS

int distill_slice_ids(int64_t n, int64_t V) {
  const int s = slice_of(n, V, kDistillSliceMost, 2048);
  // at most 64 slices: one lane each when a row is joined
  const int64_t least = ((V + 63) / 64 + kSliceStep - 1) / kSliceStep * kSliceStep;
  return (int)std::max<int64_t>(s, least);
}
size_t distill_part_bytes(int64_t n, int64_t V) {
  const int64_t s = distill_slice_ids(n, V);
  return (size_t)n * (size_t)((V + s - 1) / s) * sizeof(DistillPart);
}

int check_distill(const dspark_rows* student, const dspark_teacher* t, float temperature) {
  int rc = host_check_rows(student, "student rows NULL");
  if (rc) return rc;
  if (!t) return fail(DSPARK_EINVAL, "NULL teacher");
  if (t->k_max < 0 || t->k_max > DSPARK_K_MAX) return fail(DSPARK_EINVAL, "k_max must be in [0, DSPARK_K_MAX]");
  if (!temperature_ok(temperature)) return fail(DSPARK_EINVAL, "temperature must be in [2^-100, 2^100]");
  if (student->n_rows > 0 && (!t->len || (t->k_max > 0 && (!t->ids || !t->logits))))
    return fail(DSPARK_EINVAL, "NULL teacher list");
  return DSPARK_SUCCESS;
}

int check_distill_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (!aligned16(ws)) return fail(DSPARK_EALIGN, "workspace must be 16-byte aligned");
  if (need > 0 && (!ws || ws_bytes < need)) return fail(DSPARK_EWORKSPACE, "workspace too small");
  return DSPARK_SUCCESS;
}

DistillArgs distill_args(const dspark_rows* student, const dspark_teacher* t, float temperature, void* ws) {
  DistillArgs a{};
  a.x = student->data;
  a.x_stride = student->row_stride;
  a.n = student->n_rows;
  a.V = (int)student->vocab;
  a.slice = distill_slice_ids(a.n, a.V);
  a.slices = (a.V + a.slice - 1) / a.slice;
  a.ids = t->ids;
  a.logits = t->logits;
  a.len = t->len;
  a.lse = t->lse;
  a.k_max = t->k_max;
  a.inv_t = 1.0 / (double)temperature;
  a.part = static_cast<DistillPart*>(ws);
  if (ws) a.list_status = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + distill_part_bytes(a.n, a.V));
  return a;
}

// A slice's set of ids: its bits, and for the gradient the words' first entries.
size_t distill_lds(const DistillArgs& a, bool entries) { return (entries ? 2u : 1u) * 4u * ((size_t)a.slice / 32); }

void launch_part(const DistillArgs& a, int dtype, hipStream_t s) {
  const dim3 grid = row_slice_grid(a.n, a.slices);
  const size_t lds = distill_lds(a, false);
  if (dtype == DSPARK_BF16) hipLaunchKernelGGL(distill_part_kernel<DSPARK_BF16>, grid, dim3(kSliceBS), lds, s, a);
  else hipLaunchKernelGGL(distill_part_kernel<DSPARK_F32>, grid, dim3(kSliceBS), lds, s, a);
}
// Whether each row gets one workgroup: short rows (one launch instead of two:
// 4,096 rows of 20,003 ids in bf16, loss and gradient, 84 us against 97 in
// slices), and longer ones where they fill half of the chip, or a quarter of
// it with rows that are not long (V = 129,280 in bf16, loss and gradient: 64
// rows 26 / 20 us, 128 28 / 26, 192 30 / 35, 512 62 / 72, 4,096 443 / 539;
// the loss alone 128 rows 18 / 19, 256 19 / 23, 1,280 67 / 70; 65,536 float32,
// loss and gradient: 64 rows 22 / 25).
bool by_rows(int64_t n, int64_t V) { return V <= 32768 || (V <= kRowMost && n >= (V <= 65536 ? 64 : 128)); }
// The same for the loss alone.  Long rows that together are more than the
// last-level cache stay in slices: of rows that were read side by side the
// backward call finds less there (V = 129,280, both calls, rows / slices: 640
// float32 184 / 169 us, 1,280 bf16 177 / 171, 250 bf16 52 / 56).
bool loss_by_rows(int64_t n, int64_t V, int64_t element) {
  return by_rows(n, V) && (V <= 65536 || n * V * element <= 256 << 20);
}
template <int NWV, bool GRAD>
void launch_rows_waves(const DistillArgs& a, int dtype, hipStream_t s) {
  const size_t lds = 2u * 4u * (((size_t)a.V + 31) / 32);
  const dim3 grid = grid_of(a.n), block(64 * NWV);
  if (dtype == DSPARK_BF16) hipLaunchKernelGGL(HIP_KERNEL_NAME(distill_row_kernel<DSPARK_BF16, NWV, GRAD>), grid, block, lds, s, a);
  else hipLaunchKernelGGL(HIP_KERNEL_NAME(distill_row_kernel<DSPARK_F32, NWV, GRAD>), grid, block, lds, s, a);
}
// Rows of 128 KB or more are read for the gradient by 16 waves each: half the
// rows are in work at a time, and more of them are still in the last-level
// cache when they are read again (V = 129,280, 8 / 16 waves: 1,280 bf16 rows
// 170 / 153 us, 5,120 561 / 550, 1,280 float32 335 / 295, 256 63 / 63; 40,000
// bf16 ids, 80 KB, 5,120 rows 175 / 200).  The chip holds 512 such rows: the
// second round of somewhat more leaves CUs idle, unless the rows are long
// enough to keep HBM busy all the same (V = 129,280, 8 / 16 waves: bf16 512
// rows 65 / 63 us, 520 76 / 79, 576 79 / 85, 640 84 / 90, 704 89 / 90, 768 96 /
// 95, 800 113 / 103; float32 520 151 / 144, 640 167 / 162, 768 197 / 183; 65,536
// float32 ids 640 79 / 82, 768 95 / 90, 800 105 / 98).  A third round does not
// turn it again: 1,030 bf16 rows 141 / 126, 1,100 149 / 136.
bool rows_by_16(const DistillArgs& a, int dtype) {
  const int64_t bytes = (int64_t)a.V * (dtype == DSPARK_BF16 ? 2 : 4);
  return bytes >= 128 << 10 && (a.n <= 512 || a.n > 768 || bytes >= 384 << 10);
}
template <bool GRAD>
void launch_rows(const DistillArgs& a, int dtype, hipStream_t s) {
  if (a.V <= 8192) launch_rows_waves<4, GRAD>(a, dtype, s);
  else if (GRAD && rows_by_16(a, dtype)) launch_rows_waves<GRAD ? 16 : 8, GRAD>(a, dtype, s);
  else launch_rows_waves<8, GRAD>(a, dtype, s);
}
template <bool FROM_STATS>
void launch_grad(const DistillArgs& a, int dtype, hipStream_t s) {
  const dim3 grid = row_slice_grid(a.n, a.slices);
  const size_t lds = distill_lds(a, true);
  if (dtype == DSPARK_BF16)
    hipLaunchKernelGGL(HIP_KERNEL_NAME(distill_grad_kernel<DSPARK_BF16, FROM_STATS>), grid, dim3(kSliceBS), lds, s, a);
  else
    hipLaunchKernelGGL(HIP_KERNEL_NAME(distill_grad_kernel<DSPARK_F32, FROM_STATS>), grid, dim3(kSliceBS), lds, s, a);
}

}  // namespace
}  // namespace dspark

extern "C" {

size_t dspark_distill_workspace(int64_t n_rows, int64_t vocab) {
  if (n_rows <= 0 || n_rows > (1 << 24) || vocab < 1 || vocab > DSPARK_V_MAX) return 0;
  if (vocab <= 32768) return 0;  // (by rows, however many)
  // at least distill_part_bytes(m, vocab) + 4 m for every m <= n_rows: a row
  // has at most 64 slices and at most 2,048 / m, or those of kDistillSliceMost ids
  const int64_t few = std::min<int64_t>(2048, 64 * n_rows);
  const int64_t many = n_rows * ((vocab + kDistillSliceMost - 1) / kDistillSliceMost);
  return (size_t)std::max(few, many) * sizeof(DistillPart) + 4u * (size_t)n_rows;
}

int dspark_distill(const dspark_rows* student, const dspark_teacher* teacher, float temperature, float* loss,
                   double* stats, int32_t* row_status, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_distill(student, teacher, temperature);
  if (rc) return rc;
  if (student->n_rows == 0) return DSPARK_SUCCESS;
  if (!loss || !stats || !row_status) return fail(DSPARK_EINVAL, "NULL output");
  rc = check_distill_ws(dspark_distill_workspace(student->n_rows, student->vocab), ws, ws_bytes);
  if (rc) return rc;
  DistillArgs a = distill_args(student, teacher, temperature, ws);
  a.loss = loss;
  a.stats = stats;
  a.row_status = row_status;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (loss_by_rows(a.n, a.V, student->dtype == DSPARK_BF16 ? 2 : 4)) {
    launch_rows<false>(a, student->dtype, s);
  } else {
    launch_part(a, student->dtype, s);
    hipLaunchKernelGGL(distill_join_kernel, grid_of((a.n + kSliceNW - 1) / kSliceNW), dim3(kSliceBS), 0, s, a);
  }
  return host_check_launch();
}

int dspark_distill_backward(const dspark_rows* student, const dspark_teacher* teacher, float temperature,
                            const double* stats, const int32_t* row_status, const float* grad_loss, void* grad,
                            int64_t grad_stride, void* stream) {
  int rc = check_distill(student, teacher, temperature);
  if (rc) return rc;
  rc = check_out(student, grad, student->dtype, grad_stride);
  if (rc) return rc;
  if (student->n_rows == 0) return DSPARK_SUCCESS;
  if (!stats || !row_status || !grad_loss) return fail(DSPARK_EINVAL, "NULL stats, row_status or grad_loss");
  DistillArgs a = distill_args(student, teacher, temperature, nullptr);
  a.stats_in = stats;
  a.status_in = row_status;
  a.weight = grad_loss;
  a.grad = grad;
  a.grad_stride = grad_stride;
  launch_grad<true>(a, student->dtype, static_cast<hipStream_t>(stream));
  return host_check_launch();
}

int dspark_distill_step(const dspark_rows* student, const dspark_teacher* teacher, float temperature,
                        const float* weight, float* loss, void* grad, int64_t grad_stride, int32_t* row_status,
                        void* ws, size_t ws_bytes, void* stream) {
  int rc = check_distill(student, teacher, temperature);
  if (rc) return rc;
  rc = check_out(student, grad, student->dtype, grad_stride);
  if (rc) return rc;
  if (student->n_rows == 0) return DSPARK_SUCCESS;
  if (!weight || !loss || !row_status) return fail(DSPARK_EINVAL, "NULL weight or output");
  rc = check_distill_ws(dspark_distill_workspace(student->n_rows, student->vocab), ws, ws_bytes);
  if (rc) return rc;
  DistillArgs a = distill_args(student, teacher, temperature, ws);
  a.loss = loss;
  a.row_status = row_status;
  a.weight = weight;
  a.grad = grad;
  a.grad_stride = grad_stride;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (by_rows(a.n, a.V)) {
    launch_rows<true>(a, student->dtype, s);
  } else {
    launch_part(a, student->dtype, s);
    launch_grad<false>(a, student->dtype, s);
  }
  return host_check_launch();
}

}  // extern "C"
