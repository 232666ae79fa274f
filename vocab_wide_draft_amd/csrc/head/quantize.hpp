// Quantisation to e4m3 with a scale for each block of 128 columns
// (dspark_quantize_blocks): one pass, a block's largest |x| by lane moves
// between the 16 or 32 lanes that hold it (128 rows of blocks: by a workgroup
// that holds the block), quotients as the definition has them (a true division
// by float scales, whose ties decide a value's last bit; an exact product for
// powers of two).  Memory bounds it: 1,280 bf16 rows of 129,280 columns take 78
// us with powers of two (6.3 TB/s of what is read and written; a copy reaches
// 4.7).  Calls: those rows 88 us, with float scales, and a division for each
// value, 113; float32 rows 147 and 159 (5.6 and 5.2 TB/s); 129,280 x 5,120 in blocks
// of 128 rows 360 from bf16 and 564 from float32 with either scales (5.5 and 5.9).
#pragma once
#include "../logits/slices.hpp"

namespace dspark {

struct QuantArgs {
  const void* x;
  int64_t stride, n;
  int width, cols, blocks;  // columns of x, of the values, scales of a row
  uint8_t* v;
  int64_t v_stride;
  void* s;
  int64_t s_stride, s_step;  // scales: between rows, between blocks of 128 columns
  int chunks;  // workgroups of a row
};

constexpr float kE4m3Max = 448.0f;  // 1.75 * 2^8
constexpr int kBlock = 128;

// A block's scale, and what its values are divided by or multiplied with.
template <int ST>
struct BlockScale {
  float s, inv;  // inv: powers of two only (exact)
  bool bad;
  // most: the bits of the largest |x|, which order as the values do, with infinity and NaN above them
  __device__ __forceinline__ explicit BlockScale(uint32_t most) {
    bad = most >= 0x7f800000u;
    inv = 0.0f;
    if constexpr (ST == DSPARK_SCALE_E8M0) {
      // the exponent of a, less 8, and one more where a's fraction is above 448's
      int e = (int)(most >> 23) - 8 + ((most & 0x7fffffu) > 0x600000u ? 1 : 0);
      e = e < 1 ? 1 : e;
      e = most == 0u ? 127 : e;
      s = __uint_as_float((uint32_t)e << 23);
      inv = __uint_as_float((uint32_t)(254 - e) << 23);
    } else {
      const float q = __uint_as_float(most) / kE4m3Max;
      s = most == 0u ? 1.0f : __builtin_fmaxf(q, 0x1p-126f);
    }
  }
  __device__ __forceinline__ float scaled(float x) const {
    const float y = ST == DSPARK_SCALE_E8M0 ? x * inv : x / s;
    return __builtin_amdgcn_fmed3f(y, -kE4m3Max, kE4m3Max);
  }
  // four values, rounded to the nearest even
  __device__ __forceinline__ uint32_t four(const float* x) const {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(x[0]), scaled(x[1]), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(x[2]), scaled(x[3]), w, true);
    return bad ? 0x7f7f7f7fu : (uint32_t)w;
  }
  __device__ __forceinline__ void put(void* to, int64_t i) const {
    if constexpr (ST == DSPARK_SCALE_E8M0)
      static_cast<uint8_t*>(to)[i] = bad ? 255u : (uint8_t)(__float_as_uint(s) >> 23);
    else
      static_cast<float*>(to)[i] = bad ? __builtin_nanf("") : s;
  }
};

// a vector of a row, zeros past its width
template <int DT, int N>
__device__ __forceinline__ Raw<DT, N> raw_zero(const typename El<DT>::T* row, int v, int width) {
  if (v + N <= width) return raw_whole<DT, N, true>(row, (uint32_t)v);
  Raw<DT, N> q;
#pragma unroll
  for (int l = 0; l < N; ++l) {
    const uint32_t b = v + l < width ? __float_as_uint(El<DT>::get(row, v + l)) : 0u;
    if constexpr (DT == DSPARK_F32) q.w[l] = b;
    else if (l & 1) q.w[l >> 1] |= b;
    else q.w[l >> 1] = b >> 16;
  }
  return q;
}
// the bits of the largest |x|
template <int DT, int N>
__device__ __forceinline__ uint32_t most_of(const Raw<DT, N>& q) {
  float x[N];
  unpack<DT, N>(q, x);
  uint32_t m = 0;
#pragma unroll
  for (int l = 0; l < N; ++l) {
    const uint32_t b = __float_as_uint(x[l]) & 0x7fffffffu;
    m = b > m ? b : m;
  }
  return m;
}
// over the lanes that hold a row's block: 16 of eight values, 32 of four
template <int LANES>
__device__ __forceinline__ uint32_t most_lanes(uint32_t m) {
  const auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  m = up(m, dpp_u32<0xb1, 0xf, 0xf>(m, m));   // quad_perm 1,0,3,2
  m = up(m, dpp_u32<0x4e, 0xf, 0xf>(m, m));   // quad_perm 2,3,0,1
  m = up(m, dpp_u32<0x141, 0xf, 0xf>(m, m));  // row_half_mirror
  m = up(m, dpp_u32<0x140, 0xf, 0xf>(m, m));  // row_mirror
  if constexpr (LANES == 32) m = up(m, (uint32_t)__builtin_amdgcn_ds_swizzle((int)m, 0x401f));  // the lane 16 away
  return m;
}
template <int DT, int N, int ST>
__device__ __forceinline__ void put_values(uint8_t* at, const Raw<DT, N>& q, const BlockScale<ST>& s) {
  float x[N];
  unpack<DT, N>(q, x);
  if constexpr (N == 8) *reinterpret_cast<uint2*>(at) = make_uint2(s.four(x), s.four(x + 4));
  else *reinterpret_cast<uint32_t*>(at) = s.four(x);
}

// Scales for one row's blocks: 256 threads take U vectors each of a stretch
// of a row, all of them on their way at once.
template <int DT, int ST, int U>
__global__ void __launch_bounds__(kSliceBS) quantize_rows_kernel(QuantArgs a) {
  constexpr int N = kVec<DT>, LANES = kBlock / N;
  const int64_t b = block_number(a.n * a.chunks);
  if (b < 0) return;
  const int64_t r = a.chunks == 1 ? b : (int64_t)((uint64_t)b / (uint32_t)a.chunks);
  const int c0 = (int)(b - r * a.chunks) * (U * kSliceBS * N);
  const typename El<DT>::T* row = static_cast<const typename El<DT>::T*>(a.x) + r * a.stride;
  Raw<DT, N> q[U];
#pragma unroll
  for (int u = 0; u < U; ++u) q[u] = raw_zero<DT, N>(row, c0 + (u * kSliceBS + (int)threadIdx.x) * N, a.width);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + (u * kSliceBS + (int)threadIdx.x) * N;
    const BlockScale<ST> s(most_lanes<LANES>(most_of<DT, N>(q[u])));
    if (c < a.cols) put_values<DT, N, ST>(a.v + r * a.v_stride + c, q[u], s);
    if (c % kBlock == 0 && c / kBlock < a.blocks) s.put(a.s, r * a.s_stride + c / kBlock * a.s_step);
  }
}

// Scales for blocks of 128 rows: a workgroup for each block, which it holds.
template <int DT, int ST>
__global__ void __launch_bounds__(kSliceBS) quantize_tiles_kernel(QuantArgs a) {
  constexpr int N = kVec<DT>, LANES = kBlock / N, ROWS = kSliceBS / LANES, U = kBlock / ROWS;
  __shared__ uint32_t scratch[kSliceNW];
  const int64_t b = block_number((a.n + kBlock - 1) / kBlock * a.blocks);
  if (b < 0) return;
  const int64_t rb = (int64_t)((uint64_t)b / (uint32_t)a.blocks), r0 = rb * kBlock + threadIdx.x / LANES;
  const int cb = (int)(b - rb * a.blocks), c = cb * kBlock + (int)(threadIdx.x % LANES) * N;
  Raw<DT, N> q[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u * ROWS;
    q[u] = raw_zero<DT, N>(static_cast<const typename El<DT>::T*>(a.x) + r * a.stride, c, r < a.n ? a.width : 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t o = most_of<DT, N>(q[u]);
    m = o > m ? o : m;
  }
  m = group_reduce<kSliceNW>(m, 0u, [](uint32_t x, uint32_t y) { return x > y ? x : y; }, scratch);
  const BlockScale<ST> s(m);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t r = r0 + u * ROWS;
    if (r < a.n && c < a.cols) put_values<DT, N, ST>(a.v + r * a.v_stride + c, q[u], s);
  }
  if (threadIdx.x == 0) s.put(a.s, rb * a.s_stride + cb * a.s_step);
}

}  // namespace dspark
