// What the operators on vocabulary slices share: a workgroup of 256 threads
// works on one slice of a row's ids, a vector of neighbouring logits per
// thread at a time.
#pragma once
#include "../device_common.hpp"

namespace dspark {

constexpr int kSliceBS = 256;
constexpr int kSliceNW = kSliceBS / 64;
constexpr int kSliceStep = kSliceBS * 8;  // slices are whole multiples of it
constexpr int64_t kRowsPerY = 1 << 14;    // rows of one grid line (a multiple of 8)

// The workgroup's number in a grid of `total` workgroups laid out by grid_of
// (host side); -1 past the end (uniform).
__device__ __forceinline__ int64_t block_number(int64_t total) {
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  return b < total ? b : -1;
}

// The row and slice of a workgroup of a grid laid out by row_slice_grid: the
// slices of one row go to workgroups eight apart, which run on one of the eight
// XCDs, so that what they all read of the row stays in its L2.  False past the
// last row (uniform).
__device__ __forceinline__ bool row_slice(int64_t n, int slices, int64_t& r, int& s) {
  const uint32_t x = blockIdx.x >> 3, rows = x / (uint32_t)slices;
  s = (int)(x - rows * (uint32_t)slices);
  r = (int64_t)blockIdx.y * kRowsPerY + (int64_t)rows * 8 + (blockIdx.x & 7u);
  return r < n;
}

// a grid of `slices` workgroups for each of n rows (see row_slice; host side)
inline dim3 row_slice_grid(int64_t n, int slices) {
  const int64_t all = (n + 7) & ~int64_t(7), line = all < kRowsPerY ? all : kRowsPerY;
  return dim3((unsigned)(line * slices), (unsigned)((n + kRowsPerY - 1) / kRowsPerY));
}

typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// two binary32 values rounded to nearest even bf16 (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, r);
}

template <int DT>
struct El;
template <>
struct El<DSPARK_BF16> {
  typedef uint16_t T;
  static __device__ __forceinline__ float get(const T* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
  static __device__ __forceinline__ void put(T* p, int64_t i, float x) { p[i] = (T)(bf16_pair(x, x) & 0xffffu); }
};
template <>
struct El<DSPARK_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(const T* p, int64_t i) { return p[i]; }
  static __device__ __forceinline__ void put(T* p, int64_t i, float x) { p[i] = x; }
};

// N neighbouring logits of a row, from id v on (v a multiple of N), as one
// load of a thread: N = 8 of bf16, 4 of float32, so that the lanes of a
// wave read one unbroken stretch.  (Two loads of 16 bytes at a stride of 32,
// eight float32 per thread, fetch every line twice when they are streamed.)
template <int DT, int N>
__device__ __forceinline__ void load_whole(const typename El<DT>::T* row, int v, float (&x)[N]) {
  static_assert(N == (DT == DSPARK_BF16 ? 8 : 4), "one load of 16 bytes");
  if constexpr (DT == DSPARK_F32) {
    const v4f a = *reinterpret_cast<const v4f*>(row + v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i];
  } else {
    const v4u u = *reinterpret_cast<const v4u*>(row + v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(u[i]);
      x[2 * i + 1] = bf16_hi(u[i]);
    }
  }
}
// the same at the end of a row: ids past V read as -inf and touch no memory
template <int DT, int N>
__device__ __forceinline__ void load_vec(const typename El<DT>::T* row, int v, int V, float (&x)[N]) {
  if (v + N <= V) {
    load_whole<DT, N>(row, v, x);
  } else {
#pragma unroll
    for (int l = 0; l < N; ++l) x[l] = v + l < V ? El<DT>::get(row, v + l) : -__builtin_inff();
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_vec(typename El<DT>::T* row, int v, int V, const float (&x)[N]) {
  static_assert(N == (DT == DSPARK_BF16 ? 8 : 4), "one store of 16 bytes");
  char* at = reinterpret_cast<char*>(row) + (uint32_t)v * (uint32_t)sizeof(*row);
  if (v + N <= V) {
    if constexpr (DT == DSPARK_F32) {
      const v4f a = {x[0], x[1], x[2], x[3]};
      __builtin_nontemporal_store(a, reinterpret_cast<v4f*>(at));
    } else {
      const v4u u = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
      __builtin_nontemporal_store(u, reinterpret_cast<v4u*>(at));
    }
  } else {
#pragma unroll
    for (int l = 0; l < N; ++l)
      if (v + l < V) El<DT>::put(row, v + l, x[l]);
  }
}

// A vector as it is loaded (4 of bf16, too), to be unpacked where it is used:
// a load that is to stay in flight must not be touched before.  NT: streamed,
// not read again soon.
template <int DT, int N>
struct Raw {
  uint32_t w[DT == DSPARK_F32 ? N : N / 2];
};
template <int DT, int N, bool NT>
__device__ __forceinline__ Raw<DT, N> raw_whole(const typename El<DT>::T* row, uint32_t v) {
  Raw<DT, N> q;
  const char* at = reinterpret_cast<const char*>(row) + v * (uint32_t)sizeof(*row);  // (scalar base, 32-bit offset)
  if constexpr (sizeof(q) == 16) {
    const v4u* p = reinterpret_cast<const v4u*>(at);
    const v4u u = NT ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
    for (int i = 0; i < 4; ++i) q.w[i] = u[i];
  } else {
    const v2u* p = reinterpret_cast<const v2u*>(at);
    const v2u u = NT ? __builtin_nontemporal_load(p) : *p;
    q.w[0] = u[0];
    q.w[1] = u[1];
  }
  return q;
}
template <int DT, int N, bool NT>
__device__ __forceinline__ Raw<DT, N> raw_vec(const typename El<DT>::T* row, int v, int V) {
  if (v + N <= V) return raw_whole<DT, N, NT>(row, v);
  Raw<DT, N> q;
#pragma unroll
  for (int l = 0; l < N; ++l) {
    const uint32_t b = __float_as_uint(v + l < V ? El<DT>::get(row, v + l) : -__builtin_inff());
    if constexpr (DT == DSPARK_F32) q.w[l] = b;
    else if (l & 1) q.w[l >> 1] |= b;
    else q.w[l >> 1] = b >> 16;
  }
  return q;
}
template <int DT, int N>
__device__ __forceinline__ void unpack(const Raw<DT, N>& q, float (&x)[N]) {
#pragma unroll
  for (int l = 0; l < N; ++l)
    x[l] = DT == DSPARK_F32 ? __uint_as_float(q.w[l]) : l & 1 ? bf16_hi(q.w[l >> 1]) : bf16_lo(q.w[l >> 1]);
}

// logits of one vector of a thread
template <int DT>
constexpr int kVec = DT == DSPARK_BF16 ? 8 : 4;

// Reductions over a workgroup of NWV waves (every thread calls, every thread
// gets the result; scratch: NWV values in LDS, free again after the barrier
// that the next use starts with).
template <int NWV, class T, class OP>
__device__ __forceinline__ T group_reduce(T v, T id, OP op, T* scratch) {
  v = wave_reduce(v, id, op);
  __syncthreads();
  if (lane_id() == 0) scratch[wave_id()] = v;
  __syncthreads();
  if constexpr (NWV <= 4) {
    T r = scratch[0];
#pragma unroll
    for (int w = 1; w < NWV; ++w) r = op(r, scratch[w]);
    return r;
  } else {  // (few registers: every wave reduces the waves' results)
    return wave_reduce(lane_id() < NWV ? scratch[lane_id()] : id, id, op);
  }
}

// Sum of the values of the threads before this one, over a workgroup of NWV
// waves; *total: of all.  scratch as in group_reduce.
template <int NWV, class T>
__device__ __forceinline__ T group_excl_scan(T v, T* scratch, T* total) {
  const T inc = wave_incl_scan(v);
  __syncthreads();
  if (lane_id() == 63) scratch[wave_id()] = inc;
  __syncthreads();
  T before = inc - v, all = T(0);
#pragma unroll
  for (int w = 0; w < NWV; ++w) {
    const T o = scratch[w];
    if (w < wave_id()) before += o;
    all += o;
  }
  *total = all;
  return before;
}

// A set of a slice's ids as a bitmap, with the number of the list entry that
// each word's first id has: the entry of a member is its word's number plus
// the members before it in the word (the list is ascending).
struct IdSet {
  uint32_t* bits;   // one per id
  uint32_t* first;  // one per word of bits, set where the word is not empty
  __device__ __forceinline__ void clear(int words) {
    for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0u;
  }
  // entry e has slice-local id t; prev: the id of the entry before it, relative to the same start (negative: none here)
  __device__ __forceinline__ void add(int t, int prev, uint32_t e) {
    atomicOr(&bits[t >> 5], 1u << (t & 31));
    if (prev < 0 || (prev >> 5) != (t >> 5)) first[t >> 5] = e;
  }
  template <int N>
  __device__ __forceinline__ uint32_t members(int t) const {  // among t .. t + N - 1 (t a multiple of N, N of 4 or 8)
    return (bits[t >> 5] >> (t & 31)) & ((1u << N) - 1u);
  }
  __device__ __forceinline__ uint32_t entry(int t) const {
    return first[t >> 5] + (uint32_t)__builtin_popcount(bits[t >> 5] & ((1u << (t & 31)) - 1u));
  }
};

}  // namespace dspark
