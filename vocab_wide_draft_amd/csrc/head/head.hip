// The vocabulary head in 8-bit floating point: quantisation in blocks, and
// the product that makes logit rows, or sends their gradient back (the entry
// points declared in include/dspark.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../host_checks.hpp"
#include "dspark.h"
#include "product.hpp"
#include "quantize.hpp"

namespace dspark {
namespace {

constexpr int64_t kFp8Rows = 1 << 24, kFp8Cols = 1 << 20, kFp8Stride = 1 << 22;

int check_fp8(const dspark_fp8* q, const char* what) {
  if (!q) return fail(DSPARK_EINVAL, what);
  if (q->scale_dtype != DSPARK_SCALE_F32 && q->scale_dtype != DSPARK_SCALE_E8M0)
    return fail(DSPARK_EINVAL, "scale_dtype must be F32 or E8M0");
  if (q->block_rows != 1 && q->block_rows != kBlock) return fail(DSPARK_EINVAL, "block_rows must be 1 or 128");
  if (q->n_rows < 0 || q->n_rows > kFp8Rows) return fail(DSPARK_EINVAL, "fp8 rows out of range");
  if (q->cols < 16 || q->cols > kFp8Cols || q->cols % 16 != 0)
    return fail(DSPARK_EINVAL, "fp8 cols must be a multiple of 16 in [16, 2^20]");
  if (q->row_stride < q->cols || q->row_stride > kFp8Stride) return fail(DSPARK_EINVAL, "fp8 row_stride must be in [cols, 2^22]");
  if (q->scale_stride < (q->cols + kBlock - 1) / kBlock || q->scale_stride > kFp8Cols)
    return fail(DSPARK_EINVAL, "scale_stride must be in [a row's scales, 2^20]");
  if (!aligned16(q->values) || q->row_stride % 16 != 0)
    return fail(DSPARK_EALIGN, "fp8 rows must start 16-byte aligned (values and row_stride)");
  if (q->scale_dtype == DSPARK_SCALE_F32 && (reinterpret_cast<uintptr_t>(q->scales) & 3u) != 0)
    return fail(DSPARK_EALIGN, "float scales must be 4-byte aligned");
  if (q->n_rows > 0 && (!q->values || !q->scales)) return fail(DSPARK_EINVAL, "NULL fp8 values or scales");
  return DSPARK_SUCCESS;
}

template <int DT, int ST>
void launch_quantize(QuantArgs a, int block_rows, hipStream_t s) {
  if (block_rows == kBlock) {
    hipLaunchKernelGGL(HIP_KERNEL_NAME(quantize_tiles_kernel<DT, ST>), grid_of((a.n + kBlock - 1) / kBlock * a.blocks),
                       dim3(kSliceBS), 0, s, a);
    return;
  }
  constexpr int step = kSliceBS * kVec<DT>;
  const int all = (a.cols + step - 1) / step;
  if (a.n * all >= 4096) {
    a.chunks = (all + 3) / 4;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(quantize_rows_kernel<DT, ST, 4>), grid_of(a.n * a.chunks), dim3(kSliceBS), 0, s, a);
  } else {
    a.chunks = all;
    hipLaunchKernelGGL(HIP_KERNEL_NAME(quantize_rows_kernel<DT, ST, 1>), grid_of(a.n * a.chunks), dim3(kSliceBS), 0, s, a);
  }
}

// s_step: scales between the blocks of a row
void quantize(const dspark_rows* x, const dspark_fp8* out, int64_t s_step, hipStream_t s) {
  QuantArgs a{};
  a.x = x->data;
  a.stride = x->row_stride;
  a.n = x->n_rows;
  a.width = (int)x->vocab;
  a.cols = (int)out->cols;
  a.blocks = (a.cols + kBlock - 1) / kBlock;
  a.v = static_cast<uint8_t*>(out->values);
  a.v_stride = out->row_stride;
  a.s = out->scales;
  a.s_stride = out->scale_stride;
  a.s_step = s_step;
  if (x->dtype == DSPARK_F32) {
    if (out->scale_dtype == DSPARK_SCALE_F32) launch_quantize<DSPARK_F32, DSPARK_SCALE_F32>(a, out->block_rows, s);
    else launch_quantize<DSPARK_F32, DSPARK_SCALE_E8M0>(a, out->block_rows, s);
  } else {
    if (out->scale_dtype == DSPARK_SCALE_F32) launch_quantize<DSPARK_BF16, DSPARK_SCALE_F32>(a, out->block_rows, s);
    else launch_quantize<DSPARK_BF16, DSPARK_SCALE_E8M0>(a, out->block_rows, s);
  }
}

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

int check_product_out(int64_t M, int64_t N, const void* out, int32_t dtype, int64_t stride) {
  if (dtype != DSPARK_F32 && dtype != DSPARK_BF16) return fail(DSPARK_EINVAL, "out_dtype must be F32 or BF16");
  if (stride < N) return fail(DSPARK_EINVAL, "output stride is shorter than a row");
  if (!aligned16(out) || ((stride * (dtype == DSPARK_BF16 ? 2 : 4)) & 15) != 0)
    return fail(DSPARK_EALIGN, "output rows must start 16-byte aligned (data and stride * element size)");
  if (M > 0 && N > 0 && !out) return fail(DSPARK_EINVAL, "NULL output rows");
  return DSPARK_SUCCESS;
}

// whether `bytes` bytes at p meet rows of out
bool meet(const void* p, int64_t bytes, const void* out, int64_t rows, int64_t row_bytes, int64_t stride_bytes) {
  const char *a = static_cast<const char*>(p), *b = static_cast<const char*>(out);
  return rows > 0 && bytes > 0 && a < b + (rows - 1) * stride_bytes + row_bytes && b < a + bytes;
}
int64_t fp8_bytes(const dspark_fp8* q) { return q->n_rows > 0 ? (q->n_rows - 1) * q->row_stride + q->cols : 0; }
int64_t rows_bytes(const dspark_rows* x) {
  return x->n_rows > 0 ? ((x->n_rows - 1) * x->row_stride + x->vocab) * (x->dtype == DSPARK_BF16 ? 2 : 4) : 0;
}

// bytes from the first scale to the last
int64_t scale_bytes(const dspark_fp8* q) {
  const int64_t rows = (q->n_rows + q->block_rows - 1) / q->block_rows;
  return rows > 0 ? ((rows - 1) * q->scale_stride + (q->cols + kBlock - 1) / kBlock) * (q->scale_dtype == DSPARK_SCALE_F32 ? 4 : 1) : 0;
}

enum ProductWay { kDirect, kStaged, kTiles };
struct ProductPlan {
  ProductWay way;
  int tile_m, tile_n, splits, split_steps;
  size_t bytes;
};
ProductPlan product_plan(int64_t M, int64_t N, int64_t K, bool wide) {
  const int64_t steps = (K + kBlock - 1) / kBlock;
  ProductPlan p{};
  p.tile_n = 256;
  const int64_t tiles_n = (N + 255) / 256;
  // Few rows go straight from memory while w is short, and through LDS (whole
  // lines of w at a time) where bandwidth counts, unless tiles do as well;
  // direct / staged / tiles, float scales, bf16 results, w out of the caches, us of
  // a call: 20,003 x 1,008 (20 MB), 1 row 8.4 / 11.6 / 12.6, 32 rows 11.7 / 16.3 /
  // 13.5; 60,000 x 1,008 15.7 / 18.3 / 15.7, 21 / 27 / 17; 102,000 x 1,008 24 / 26 /
  // 28, 33 / 31 / 30; 129,280 x 1,024 (132 MB) 27 / 27 / 28, 37 / 30 / 30; 40,000 x
  // 5,120 (205 MB) 49 / 41 / 43, 69 / 51 / 49; 129,280 x 5,120 128 / 113 / 113,
  // 184 / 122 / 121.  Longer rows would have the border lower than the bytes do:
  // 4,000 x 5,120 11.3 / 12.9 / 13.4, 14.4 / 17.0 / 15.7; 12,000 x 5,120 20 / 18 / 17,
  // 28 / 24 / 19; 20,000 x 5,120 (102 MB) 32 / 25 / 24, 46 / 32 / 27.  float32 results
  // of 17 rows and more stay staged, as tiles have the slower instruction: 32 rows of
  // 129,280 x 1,024 33.7 / 36.4 (staged / tiles), 40,000 x 5,120 52 / 56, 129,280 x
  // 5,120 130 / 144.
  const int64_t bytes = N * K;
  const bool direct = M <= 32 && bytes <= 112 << 20;
  if (direct || M <= 16 || (M <= 32 && (wide || bytes > 300 << 20))) {
    p.way = direct ? kDirect : kStaged;
    p.tile_m = M <= 16 ? 16 : 32;
    if (direct) p.tile_n = 64;
    const int64_t tiles = (N + p.tile_n - 1) / p.tile_n;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(tiles, 1), steps / 4));
    p.split_steps = (int)((steps + want - 1) / want);
  } else {
    // The width and the number of parts that should take least: rounds of 256
    // tiles (parts of a long product fill the last one); for a step of a tile of
    // 64 u rows 0.38 + 0.28 u us, and 0.86 us for its columns of w out of memory
    // shared by the tiles that read them; three steps for a tile's beginning and
    // end; the parts' way through memory.  (129,280 x 5,120, powers of two, us for
    // u = 1, 2, 3, 4, the last tile as narrow as what is left: 64 rows 129, 127, 127,
    // 127; 128: 184, 144, 144, 144; 256: 304, 223, 223, 194; 384: 400, 306, 262, 276;
    // 768: 753, 547, 482, 447; 5,120: 4,623, 3,315, 3,021, 2,700.)  The constants are
    // fitted to these.  Float scales, and float32 results with twice the time of
    // matrix instructions, order the choices alike (float scales, u = 1, 2, 3, 4: 384
    // rows 443, 339, 298, 308; 5,120 5,280, 3,906, 3,486, 3,191; float32 results, u =
    // 1, 2: 64 rows 149, 152; 128: 259, 203; 384: 701, 532; 5,120: 8,870, 6,528; a
    // gradient, 384 rows x 5,120 x 129,280, u = 2 in 4, 6, 8, 12, 16 parts 543, 623,
    // 530, 546, 539, the rule's 518): its choice is within 3 % of the best of those.
    p.way = kTiles;
    double best = 0.0;
    for (int u = wide ? 2 : 4; u >= 1; --u) {
      const int64_t tiles_m = (M + 64 * u - 1) / (64 * u), tiles = tiles_m * tiles_n;
      for (int64_t s = 1; s <= 16 && (s == 1 || (steps / s >= 8 && tiles * (s - 1) < 1024)); ++s) {
        const double rounds = (double)(tiles * s) / 256.0;
        const double time = (rounds < 8.0 ? std::ceil(rounds) : rounds) * (double)((steps + s - 1) / s + 3) *
                                (0.38 + 0.28 * u + 0.86 / (double)tiles_m) +
                            (s > 1 ? 2e-6 * 4.0 * (double)s * (double)M * (double)N / 4.0 : 0.0);
        if (best == 0.0 || time < best) {
          best = time;
          p.tile_m = 64 * u;
          p.split_steps = (int)((steps + s - 1) / s);
        }
      }
    }
  }
  p.splits = (int)((steps + p.split_steps - 1) / p.split_steps);
  p.bytes = p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)up(N, 4) * 4u : 0;
  return p;
}

// whichever type the results have
size_t product_bytes(int64_t M, int64_t N, int64_t K) {
  return std::max(product_plan(M, N, K, false).bytes, product_plan(M, N, K, true).bytes);
}

// The same for any number of rows up to M: where a long product has fewer
// parts with more rows, fewer rows take more.  Among as many 64s of rows (which
// is all that a plan's tiles and their cost hang on, but for the parts' way
// through memory, which grows with the rows) the first has the most parts.
size_t most_product_bytes(int64_t M, int64_t N, int64_t K) {
  const int64_t steps = (K + kBlock - 1) / kBlock, tiles_n = (N + 255) / 256, row_bytes = up(N, 4) * 4;
  size_t most = std::max({product_bytes(M, N, K), product_bytes(std::min<int64_t>(M, 16), N, K), product_bytes(std::min<int64_t>(M, 32), N, K)});
  int64_t last = 0;
  for (int64_t first = 17; first <= M; first = last + 1) {
    last = std::min(first == 17 ? 32 : up(first, 64), M);  // (17 to 32 rows: tiles only for some lengths of w)
    const int64_t tiles = (first + 255) / 256 * tiles_n;  // (of the largest ones)
    const int64_t parts = std::min<int64_t>({16, steps / 8, 1 + 1023 / tiles});
    if (parts < 2 && first > 17) break;
    if ((size_t)(parts * last * row_bytes) <= most) continue;
    const int splits = std::max(product_plan(first, N, K, false).splits, product_plan(first, N, K, true).splits);
    if (splits > 1) most = std::max(most, (size_t)(splits * last * row_bytes));
  }
  return most;
}

template <int ST, bool WIDE, int OUT, int U>
void launch_tile(const ProductArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(HIP_KERNEL_NAME(product_tile_kernel<U, ST, WIDE, OUT>), grid_of(a.tiles_m * a.tiles_n * a.splits),
                     dim3(512), 0, s, a);
}
template <int ST, bool WIDE, int OUT>
void launch_tiles(const ProductPlan& p, ProductArgs a, hipStream_t s) {
  const dim3 grid = grid_of(a.tiles_m * a.tiles_n * a.splits);
  if (p.way == kDirect) {
    if (p.tile_m == 16) hipLaunchKernelGGL(HIP_KERNEL_NAME(product_direct_kernel<1, ST, WIDE, OUT>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(product_direct_kernel<2, ST, WIDE, OUT>), grid, dim3(256), 0, s, a);
    return;
  }
  if (p.way == kStaged) {
    if (p.tile_m == 16) hipLaunchKernelGGL(HIP_KERNEL_NAME(product_staged_kernel<1, ST, WIDE, OUT>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(HIP_KERNEL_NAME(product_staged_kernel<2, ST, WIDE, OUT>), grid, dim3(256), 0, s, a);
    return;
  }
  if (p.tile_m == 64) launch_tile<ST, WIDE, OUT, 1>(a, s);
  else if (p.tile_m == 128) launch_tile<ST, WIDE, OUT, 2>(a, s);
  if constexpr (!WIDE) {
    if (p.tile_m == 192) launch_tile<ST, WIDE, OUT, 3>(a, s);
    else if (p.tile_m == 256) launch_tile<ST, WIDE, OUT, 4>(a, s);
  }
}

void product(const dspark_fp8* x, int64_t xs_step, const dspark_fp8* w, void* out, int32_t out_dtype, int64_t out_stride, void* ws, hipStream_t s) {
  const ProductPlan p = product_plan(x->n_rows, w->n_rows, x->cols, out_dtype == DSPARK_F32);
  ProductArgs a{};
  a.x = static_cast<const uint8_t*>(x->values);
  a.w = static_cast<const uint8_t*>(w->values);
  a.x_stride = x->row_stride;
  a.w_stride = w->row_stride;
  a.xs = x->scales;
  a.ws = w->scales;
  a.xs_stride = x->scale_stride;
  a.xs_step = xs_step;
  a.ws_stride = w->scale_stride;
  a.M = x->n_rows;
  a.N = w->n_rows;
  a.K = (int)x->cols;
  a.steps = (a.K + kBlock - 1) / kBlock;
  a.splits = p.splits;
  a.split_steps = p.split_steps;
  a.tiles_m = (a.M + p.tile_m - 1) / p.tile_m;
  a.tiles_n = (a.N + p.tile_n - 1) / p.tile_n;
  a.out = p.splits > 1 ? ws : out;
  a.out_stride = p.splits > 1 ? up(a.N, 4) : out_stride;
  const bool wide = out_dtype == DSPARK_F32, bf16 = p.splits == 1 && !wide;
  if (x->scale_dtype == DSPARK_SCALE_F32) {
    if (wide) launch_tiles<DSPARK_SCALE_F32, true, DSPARK_F32>(p, a, s);
    else if (bf16) launch_tiles<DSPARK_SCALE_F32, false, DSPARK_BF16>(p, a, s);
    else launch_tiles<DSPARK_SCALE_F32, false, DSPARK_F32>(p, a, s);
  } else {
    if (wide) launch_tiles<DSPARK_SCALE_E8M0, true, DSPARK_F32>(p, a, s);
    else if (bf16) launch_tiles<DSPARK_SCALE_E8M0, false, DSPARK_BF16>(p, a, s);
    else launch_tiles<DSPARK_SCALE_E8M0, false, DSPARK_F32>(p, a, s);
  }
  if (p.splits > 1) {
    ProductJoinArgs j{};
    j.part = static_cast<const float*>(ws);
    j.splits = p.splits;
    j.vectors = (int)(a.out_stride / 4);
    j.M = a.M;
    j.N = a.N;
    j.out = out;
    j.out_stride = out_stride;
    const dim3 grid = grid_of((j.M * j.vectors + kSliceBS - 1) / kSliceBS);
    if (out_dtype == DSPARK_F32) hipLaunchKernelGGL(product_join_kernel<DSPARK_F32>, grid, dim3(kSliceBS), 0, s, j);
    else hipLaunchKernelGGL(product_join_kernel<DSPARK_BF16>, grid, dim3(kSliceBS), 0, s, j);
  }
}

bool product_sizes(int64_t M, int64_t N, int64_t cols) {
  return M > 0 && M <= kFp8Rows && N > 0 && N <= kFp8Rows && cols >= 1 && cols <= kFp8Cols;
}

// The quantised rows of a linear call in its workspace: values, scales, and
// behind them the product's.
struct LinearPlan {
  int64_t cols, blocks;
  size_t scales_at, ws_at, bytes;
};
LinearPlan linear_plan(int64_t M, int64_t N, int64_t width) {
  LinearPlan p{};
  p.cols = up(width, 16);
  p.blocks = (p.cols + kBlock - 1) / kBlock;
  p.scales_at = (size_t)(M * p.cols);
  p.ws_at = p.scales_at + (size_t)up(M * p.blocks * 4, 256);
  p.bytes = p.ws_at + product_bytes(M, N, p.cols);
  return p;
}

int check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (!aligned16(ws)) return fail(DSPARK_EALIGN, "workspace must be 16-byte aligned");
  if (need > 0 && (!ws || ws_bytes < need)) return fail(DSPARK_EWORKSPACE, "workspace too small");
  return DSPARK_SUCCESS;
}

// whether a workspace of `bytes` bytes meets a matrix
bool meets(const void* ws, size_t bytes, const dspark_fp8* q) {
  return meet(ws, (int64_t)bytes, q->values, q->n_rows, q->cols, q->row_stride) || meet(ws, (int64_t)bytes, q->scales, 1, scale_bytes(q), 0);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" {

int dspark_quantize_blocks(const dspark_rows* x, const dspark_fp8* out, void* stream) {
  int rc = host_check_rows(x, "rows NULL");
  if (rc) return rc;
  rc = check_fp8(out, "NULL fp8 matrix");
  if (rc) return rc;
  if (out->n_rows != x->n_rows) return fail(DSPARK_EINVAL, "the fp8 matrix has another number of rows");
  if (out->cols != up(x->vocab, 16)) return fail(DSPARK_EINVAL, "fp8 cols must be the rows' width rounded up to a multiple of 16");
  if (x->n_rows == 0) return DSPARK_SUCCESS;
  if (meet(x->data, rows_bytes(x), out->values, out->n_rows, out->cols, out->row_stride) ||
      meet(x->data, rows_bytes(x), out->scales, 1, scale_bytes(out), 0))
    return fail(DSPARK_EINVAL, "the fp8 matrix overlaps the rows");
  if (meet(out->scales, scale_bytes(out), out->values, out->n_rows, out->cols, out->row_stride))
    return fail(DSPARK_EINVAL, "the fp8 matrix's scales overlap its values");
  quantize(x, out, 1, static_cast<hipStream_t>(stream));
  return host_check_launch();
}

size_t dspark_block_product_workspace(int64_t x_rows, int64_t w_rows, int64_t cols) {
  return product_sizes(x_rows, w_rows, cols) ? most_product_bytes(x_rows, w_rows, up(cols, 16)) : 0;
}

int dspark_block_product(const dspark_fp8* x, const dspark_fp8* w, void* out, int32_t out_dtype, int64_t out_stride,
                         void* ws, size_t ws_bytes, void* stream) {
  int rc = check_fp8(x, "NULL left matrix");
  if (rc) return rc;
  rc = check_fp8(w, "NULL right matrix");
  if (rc) return rc;
  if (x->block_rows != 1 || w->block_rows != kBlock) return fail(DSPARK_EINVAL, "block_rows must be 1 on the left and 128 on the right");
  if (x->cols != w->cols) return fail(DSPARK_EINVAL, "the matrices' cols differ");
  if (x->scale_dtype != w->scale_dtype) return fail(DSPARK_EINVAL, "the matrices' scale_dtype differs");
  rc = check_product_out(x->n_rows, w->n_rows, out, out_dtype, out_stride);
  if (rc) return rc;
  if (x->n_rows == 0 || w->n_rows == 0) return DSPARK_SUCCESS;
  const int64_t es = out_dtype == DSPARK_BF16 ? 2 : 4;
  if (meet(x->values, fp8_bytes(x), out, x->n_rows, w->n_rows * es, out_stride * es) ||
      meet(w->values, fp8_bytes(w), out, x->n_rows, w->n_rows * es, out_stride * es) ||
      meet(x->scales, scale_bytes(x), out, x->n_rows, w->n_rows * es, out_stride * es) ||
      meet(w->scales, scale_bytes(w), out, x->n_rows, w->n_rows * es, out_stride * es))
    return fail(DSPARK_EINVAL, "output rows overlap an input");
  const size_t need = product_bytes(x->n_rows, w->n_rows, x->cols);
  rc = check_ws(need, ws, ws_bytes);
  if (rc) return rc;
  if (meets(ws, need, x) || meets(ws, need, w) || meet(ws, (int64_t)need, out, x->n_rows, w->n_rows * es, out_stride * es))
    return fail(DSPARK_EINVAL, "the workspace overlaps an input or the output");
  product(x, 1, w, out, out_dtype, out_stride, ws, static_cast<hipStream_t>(stream));
  return host_check_launch();
}

size_t dspark_block_linear_workspace(int64_t x_rows, int64_t w_rows, int64_t cols) {
  return product_sizes(x_rows, w_rows, cols) ? linear_plan(x_rows, w_rows, cols).ws_at + most_product_bytes(x_rows, w_rows, up(cols, 16)) : 0;
}

int dspark_block_linear(const dspark_rows* x, const dspark_fp8* w, void* out, int32_t out_dtype, int64_t out_stride,
                        void* ws, size_t ws_bytes, void* stream) {
  int rc = host_check_rows(x, "rows NULL");
  if (rc) return rc;
  rc = check_fp8(w, "NULL right matrix");
  if (rc) return rc;
  if (w->block_rows != kBlock) return fail(DSPARK_EINVAL, "block_rows must be 128 on the right");
  if (w->cols != up(x->vocab, 16)) return fail(DSPARK_EINVAL, "w->cols must be the rows' width rounded up to a multiple of 16");
  rc = check_product_out(x->n_rows, w->n_rows, out, out_dtype, out_stride);
  if (rc) return rc;
  if (x->n_rows == 0 || w->n_rows == 0) return DSPARK_SUCCESS;
  const int64_t es = out_dtype == DSPARK_BF16 ? 2 : 4;
  if (meet(x->data, rows_bytes(x), out, x->n_rows, w->n_rows * es, out_stride * es) ||
      meet(w->values, fp8_bytes(w), out, x->n_rows, w->n_rows * es, out_stride * es) ||
      meet(w->scales, scale_bytes(w), out, x->n_rows, w->n_rows * es, out_stride * es))
    return fail(DSPARK_EINVAL, "output rows overlap an input");
  const LinearPlan p = linear_plan(x->n_rows, w->n_rows, x->vocab);
  rc = check_ws(p.bytes, ws, ws_bytes);
  if (rc) return rc;
  if (meet(ws, (int64_t)p.bytes, x->data, 1, rows_bytes(x), 0) || meets(ws, p.bytes, w) ||
      meet(ws, (int64_t)p.bytes, out, x->n_rows, w->n_rows * es, out_stride * es))
    return fail(DSPARK_EINVAL, "the workspace overlaps an input or the output");
  char* at = static_cast<char*>(ws);
  // (its scales by blocks: a tile's rows lie next to each other)
  dspark_fp8 q{at, at + p.scales_at, w->scale_dtype, 1, x->n_rows, p.cols, p.cols, 1};
  hipStream_t s = static_cast<hipStream_t>(stream);
  quantize(x, &q, x->n_rows, s);
  product(&q, x->n_rows, w, out, out_dtype, out_stride, p.bytes > p.ws_at ? at + p.ws_at : nullptr, s);
  return host_check_launch();
}

}  // extern "C"
