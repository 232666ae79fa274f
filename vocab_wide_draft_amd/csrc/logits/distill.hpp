// Distillation loss against a teacher's top logits, and its gradient
// (dspark_distill, dspark_distill_backward, dspark_distill_step).
//
// Mathematics.  u = s / T.  Off the list, a row needs M_off = max s and S_off =
// sum exp(u - M_off / T); on the list M_on and S_on, and, with w_j = exp(z_j / T
// - zm) (zm: the teacher's lse, or the list's maximum when it is
// renormalised), B0 = sum w_j and B1 = sum w_j (z_j / T - zm - (u_j - M / T)),
// M the row's maximum: a row far from zero, such as one that a mask has left
// at its type's lowest value, would lose its loss in the difference of two
// sums of the logits themselves.  The two sides are kept apart, each with its
// own maximum: S - S_on would cancel where the list holds nearly all mass, and
// with one maximum S_off would underflow where the list lies far above the
// rest, while the loss still holds the logarithm of that mass and the gradient
// its distribution.  With M = max(M_off, M_on) and
// S = S_off e^((M_off - M) / T) + S_on e^((M_on - M) / T),
//   log Q = (M_off - M) / T + log S_off - log S
//   with lse:    loss = B1 + B0 log S + P (log P - log Q),  P = 1 - B0
//                off the list dL/du_v = e^(u_v - M_off / T) (e^((M_off - M) / T) / S - P / S_off)
//   normalised:  loss = B1 / B0 - log B0 + log S  (every id counts as off the list in the sums)
// The softmax stands in the gradient times sum p, which is B0 with lse and one
// otherwise.  The last term adds P to it, B0 + P = 1; without that term (P <= 0,
// or nothing off the list) the factor stays, and 1 / S is kept as B0 / S.
// Every term is a sum over slices of the vocabulary once each slice's maximum
// is put back (in B1, too), so slices are worked on apart and joined.  Sums
// over a thread's logits are binary32, everything joined is binary64, as is the
// list's side (P = 1 - B0 loses what binary32 would keep of it).  The hardware
// exponential gives 0 below 2^-126 relative to a maximum.
#pragma once
#include "slices.hpp"

namespace dspark {

struct DistillPart {  // one slice of one row
  double s_off, s_on, b0, b1, zm;
  float m_off, m_on;
  int32_t flags;  // 1: a NaN, 2: a +inf
  int32_t reserved;
};

struct DistillArgs {
  const void* x;
  int64_t x_stride;
  int64_t n;
  int V;
  int slices, slice;
  const int32_t* ids;
  const float* logits;
  const int32_t* len;
  const float* lse;
  int k_max;
  double inv_t;
  DistillPart* part;  // [n][slices]
  int32_t* list_status;  // [n] (the list's refusal)
  float* loss;
  double* stats;
  int32_t* row_status;
  const int32_t* status_in;  // backward
  const double* stats_in;
  const float* weight;
  void* grad;
  int64_t grad_stride;
};

constexpr int kListPer = DSPARK_K_MAX / kSliceBS;  // list entries per thread
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ bool finite_row_value(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// body(t, v) for every vector of a row's ids [start, start + size) that this
// thread of T owns, t counted from start; kAhead loads are on their way at a
// time (5,120 bf16 rows, loss and gradient: 550 us, as with 2; 6 628 and 8
// 665: more registers, fewer waves).  LAST: streamed, the row is not read
// again (a first reading that is streamed too leaves less in the caches for
// the second: 670 us).
constexpr int kAhead = 4;
template <int DT, bool LAST, int T, class BODY>
__device__ __forceinline__ void for_row(const typename El<DT>::T* x, int start, int size, BODY body) {
  constexpr int N = kVec<DT>, STEP = T * N;
  const typename El<DT>::T* row = x + start;
  const int whole = size / (kAhead * STEP) * (kAhead * STEP);
  for (int base = 0; base < whole; base += kAhead * STEP) {
    Raw<DT, N> q[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) q[k] = raw_whole<DT, N, LAST>(row, (uint32_t)(base + k * STEP + (int)threadIdx.x * N));
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      float v[N];
      unpack<DT, N>(q[k], v);
      body(base + k * STEP + (int)threadIdx.x * N, v);
    }
  }
  if (whole == size) return;
  Raw<DT, N> q[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int t = whole + k * STEP + (int)threadIdx.x * N;
    if (t < size) q[k] = raw_vec<DT, N, LAST>(row, t, size);
  }
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int t = whole + k * STEP + (int)threadIdx.x * N;
    if (t < size) {
      float v[N];
      unpack<DT, N>(q[k], v);
      body(t, v);
    }
  }
}

// The slice's part of a row (see above).  Returns with the whole workgroup.
template <int DT>
__device__ void distill_slice(const DistillArgs& a, int64_t r, int s, uint32_t* lds) {
  __shared__ double red[kSliceNW];
  __shared__ float redf[kSliceNW];
  __shared__ uint32_t redu[kSliceNW];
  typedef typename El<DT>::T XT;
  const int start = s * a.slice, V = a.V;
  const int size = V - start < a.slice ? V - start : a.slice;
  const int words = (a.slice + 31) / 32;
  const XT* x = static_cast<const XT*>(a.x) + r * a.x_stride;
  const int32_t* ids = a.ids + r * a.k_max;
  const float* zl = a.logits + r * a.k_max;
  int len = a.len[r];
  uint32_t wrong = 0;
  if (len < 0 || len > a.k_max) {
    wrong = 1u;
    len = 0;
  }
  const bool tail = a.lse != nullptr;
  IdSet on{lds, nullptr};  // (members alone are asked for)
  if (len > 0 && tail) on.clear(words);
  // the list: which entries are ours, and (slice 0) whether it may be used
  int32_t id[kListPer];
  float z[kListPer];
  float zmax = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < kListPer; ++j) {
    const int e = j * kSliceBS + (int)threadIdx.x;
    id[j] = -1;
    z[j] = -__builtin_inff();
    if (e < len) {
      id[j] = ids[e];
      z[j] = zl[e];
      zmax = __builtin_fmaxf(zmax, z[j]);
      if (s == 0) {
        if ((uint32_t)id[j] >= (uint32_t)V) wrong |= 2u;
        if (e > 0 && ids[e - 1] >= id[j]) wrong |= 4u;
        if (!finite_row_value(z[j])) wrong |= 8u;
      }
    }
  }
  if (s == 0) {
    if (len > 0 && tail && !finite_row_value(a.lse[r])) wrong |= 8u;
    wrong = group_reduce<kSliceNW>(wrong, 0u, [](uint32_t p, uint32_t q) { return p | q; }, redu);
    if (threadIdx.x == 0) a.list_status[r] = wrong ? DSPARK_ST_Q_BAD_LEN + (wrong & 1u ? 0 : wrong & 2u ? 1 : wrong & 4u ? 2 : 3) : DSPARK_ST_OK;
  }
  if (len == 0) return;  // (uniform)
  double zm;
  if (tail) {
    zm = (double)a.lse[r];
  } else {
    zm = (double)group_reduce<kSliceNW>(zmax, -__builtin_inff(), [](float p, float q) { return __builtin_fmaxf(p, q); }, redf) * a.inv_t;
  }
  __syncthreads();
  const float c = (float)(a.inv_t * (double)kLog2e);
  if (tail) {
#pragma unroll
    for (int j = 0; j < kListPer; ++j) {
      const uint32_t t = (uint32_t)(id[j] - start);
      if (id[j] >= 0 && t < (uint32_t)size) atomicOr(&on.bits[t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  // the row off the list: running maximum and sum; a vector moves the maximum
  // at most once
  constexpr int N = kVec<DT>;
  uint32_t flags = 0;
  float m = -__builtin_inff(), s_off = 0.0f;
  for_row<DT, false, kSliceBS>(x, start, size, [&](int t, float (&v)[N]) {
    const uint32_t bits = tail ? on.members<N>(t) : 0u;
    if (bits) {
#pragma unroll
      for (int l = 0; l < N; ++l) v[l] = (bits >> l) & 1u ? -__builtin_inff() : v[l];
    }
    float top = v[0];
#pragma unroll
    for (int l = 1; l < N; ++l) top = __builtin_fmaxf(top, v[l]);
    if (top > m) {
      s_off *= __builtin_amdgcn_exp2f((m - top) * c);  // (by 0 the first time)
      m = top;
    }
    const float ref = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int l = 0; l < N; ++l) s_off += __builtin_amdgcn_exp2f((v[l] - ref) * c);
  });
  // a NaN or +inf shows in the sum or the maximum; which of the two, the thread's own logits tell
  if (s_off != s_off || m == __builtin_inff()) {
    for (int t = threadIdx.x * N; t < size; t += kSliceBS * N) {
      float v[N];
      load_vec<DT, N>(x, start + t, V, v);
#pragma unroll
      for (int l = 0; l < N; ++l) flags |= v[l] != v[l] ? 1u : v[l] == __builtin_inff() ? 2u : 0u;
    }
  }
  // the list's side, now that the slice is in the caches
  double b0 = 0.0, b1 = 0.0;
  float m_own = -__builtin_inff(), s_on = 0.0f, x_list[kListPer];
#pragma unroll
  for (int j = 0; j < kListPer; ++j) {
    const uint32_t t = (uint32_t)(id[j] - start);
    x_list[j] = -__builtin_inff();
    if (id[j] >= 0 && t < (uint32_t)size) {
      const float xj = x_list[j] = El<DT>::get(x, id[j]);
      m_own = __builtin_fmaxf(m_own, xj);
      if (tail) flags |= xj != xj ? 1u : xj == __builtin_inff() ? 2u : 0u;
    } else {
      id[j] = -1;
    }
  }
  // b1 from this thread's largest listed logit first: once the slice's maximum
  // is known, one addition puts it back
  const double ref = m_own == -__builtin_inff() ? 0.0 : (double)m_own;
#pragma unroll
  for (int j = 0; j < kListPer; ++j) {
    if (id[j] >= 0) {
      const double lp = (double)z[j] * a.inv_t - zm;
      const double w = exp(lp);
      if (w > 0.0) {
        b0 += w;
        b1 += w * (lp - ((double)x_list[j] - ref) * a.inv_t);
      }
    }
  }
  const float m_on = tail ? m_own : -__builtin_inff();
  if (m_on > -__builtin_inff()) {
#pragma unroll
    for (int j = 0; j < kListPer; ++j) s_on += __builtin_amdgcn_exp2f((x_list[j] - m_on) * c);
  }
  const auto larger = [](float p, float q) { return __builtin_fmaxf(p, q); };
  const auto plus = [](double p, double q) { return p + q; };
  const float M_off = group_reduce<kSliceNW>(m, -__builtin_inff(), larger, redf);
  const float M_on = group_reduce<kSliceNW>(m_on, -__builtin_inff(), larger, redf);
  const float M = __builtin_fmaxf(M_off, M_on);
  if (b0 > 0.0 && M > -__builtin_inff()) b1 += b0 * (((double)M - ref) * a.inv_t);  // (without a finite logit b1 is +inf)
  flags = group_reduce<kSliceNW>(flags, 0u, [](uint32_t p, uint32_t q) { return p | q; }, redu);
  const double f = m == -__builtin_inff() ? 0.0 : (double)__builtin_amdgcn_exp2f((m - M_off) * c);
  const double g = m_on == -__builtin_inff() ? 0.0 : (double)__builtin_amdgcn_exp2f((m_on - M_on) * c);
  const double t_off = group_reduce<kSliceNW>((double)s_off * f, 0.0, plus, red);
  const double t_on = group_reduce<kSliceNW>((double)s_on * g, 0.0, plus, red);
  b0 = group_reduce<kSliceNW>(b0, 0.0, plus, red);
  b1 = group_reduce<kSliceNW>(b1, 0.0, plus, red);
  if (threadIdx.x == 0) {
    DistillPart& p = a.part[r * a.slices + s];
    p.s_off = t_off;
    p.s_on = t_on;
    p.b0 = b0;
    p.b1 = b1;
    p.zm = zm;
    p.m_off = M_off;
    p.m_on = M_on;
    p.flags = (int32_t)flags;
    p.reserved = 0;
  }
}

struct DistillRow {  // what the gradient needs of a row
  int status;
  double M;      // the row's maximum
  double inv_s;  // 1 / S, times sum p where the last term is left out
  double M_off;  // the maximum off the list
  double f_off;  // dL/du off the list over e^(u - M_off / T)
  double zm;     // log of the teacher's normaliser
  double loss;
};

// Status of a good list's row from its sums and flags.  With lse, listed
// probabilities that sum to more than binary32 holds are the list's fault: lse
// far too small, as its 24 bits may make it at low temperatures.
__device__ __forceinline__ int distill_status(bool tail, double b0, uint32_t flags, float m) {
  return tail && !(b0 <= (double)3.40282347e38f) ? DSPARK_ST_Q_NONFINITE
         : flags & 1u ? DSPARK_ST_ROW_NAN
         : flags & 2u ? DSPARK_ST_ROW_POSINF
         : m == -__builtin_inff() ? DSPARK_ST_ROW_ZERO_MASS : DSPARK_ST_OK;
}

// The loss and the gradient's numbers from a row's sums (a finite maximum, which b1 is relative to, no NaN, no +inf).
__device__ __forceinline__ void distill_finish(double inv_t, bool tail, float m_off, float m_on, double off, double on,
                                               double b0, double b1, double zm, DistillRow& o) {
  constexpr float kNone = -__builtin_inff();
  const float m = __builtin_fmaxf(m_off, m_on);
  // e^((x - m) / T), 0 where x is none
  const double e_off = m_off == kNone ? 0.0 : exp(((double)m_off - (double)m) * inv_t);
  const double e_on = m_on == kNone ? 0.0 : exp(((double)m_on - (double)m) * inv_t);
  const double S = off * e_off + on * e_on;  // (the first underflows where the rest is out of sight)
  const double log_s = log(S);
  o.M = m;
  o.M_off = m_off == kNone ? 0.0 : m_off;
  const double P = 1.0 - b0;
  const bool rest = tail && P > 0.0 && off > 0.0;  // the last term
  o.inv_s = (tail && !rest ? b0 : 1.0) / S;
  o.f_off = e_off * o.inv_s;
  if (tail) {
    o.zm = zm;
    o.loss = b1 + b0 * log_s;
    if (rest) {
      o.loss += P * (log(P) - (((double)m_off - (double)m) * inv_t + log(off) - log_s));
      o.f_off -= P / off;
    }
  } else {
    const double lz = log(b0);
    o.zm = zm + lz;
    o.loss = b1 / b0 - lz + log_s;
  }
}

// One wave joins the slices of a row (every lane gets the result).
__device__ __forceinline__ DistillRow distill_join(const DistillArgs& a, int64_t r) {
  DistillRow o{a.list_status[r], 0.0, 0.0, 0.0, 0.0, 0.0, 0.0};
  if (o.status != DSPARK_ST_OK || a.len[r] == 0) return o;
  const int l = lane_id();
  constexpr float kNone = -__builtin_inff();
  DistillPart p{0.0, 0.0, 0.0, 0.0, 0.0, kNone, kNone, 0, 0};
  if (l < a.slices) p = a.part[r * a.slices + l];
  const auto larger = [](float x, float y) { return __builtin_fmaxf(x, y); };
  const uint32_t flags = wave_reduce((uint32_t)p.flags, 0u, [](uint32_t x, uint32_t y) { return x | y; });
  const float m_off = wave_reduce(p.m_off, kNone, larger), m_on = wave_reduce(p.m_on, kNone, larger);
  const float m = __builtin_fmaxf(m_off, m_on);
  const double b0 = wave_sum(p.b0);
  o.status = distill_status(a.lse != nullptr, b0, flags, m);
  if (o.status != DSPARK_ST_OK) return o;
  // e^((x - y) / T) of two maxima, 0 where x is none
  const auto shift = [&](float x, float y) { return x == kNone ? 0.0 : exp(((double)x - (double)y) * a.inv_t); };
  const double off = wave_sum(p.s_off * shift(p.m_off, m_off)), on = wave_sum(p.s_on * shift(p.m_on, m_on));
  // a slice's maximum put back in b1, to which it adds: no difference of large numbers
  const float m_own = __builtin_fmaxf(p.m_off, p.m_on);
  const double lower = m_own == kNone ? 0.0 : ((double)m - (double)m_own) * a.inv_t;
  const double b1 = wave_sum(p.b1 + p.b0 * lower);
  distill_finish(a.inv_t, a.lse != nullptr, m_off, m_on, off, on, b0, b1, a.part[r * a.slices].zm, o);
  return o;
}

__device__ __forceinline__ void distill_row_out(const DistillArgs& a, int64_t r, const DistillRow& o) {
  a.loss[r] = (float)o.loss;
  a.row_status[r] = o.status;
  if (a.stats) {
    double* st = a.stats + r * DSPARK_DISTILL_STATS;
    st[0] = o.M;
    st[1] = o.inv_s;
    st[2] = o.M_off;
    st[3] = o.f_off;
    st[4] = o.zm;
  }
}

template <int DT>
__global__ void __launch_bounds__(kSliceBS) distill_part_kernel(DistillArgs a) {
  extern __shared__ uint32_t lds[];
  int64_t r;
  int s;
  if (!row_slice(a.n, a.slices, r, s)) return;
  distill_slice<DT>(a, r, s, lds);
}

// one wave per row
__global__ void __launch_bounds__(kSliceBS) distill_join_kernel(DistillArgs a) {
  const int64_t b = block_number((a.n + kSliceNW - 1) / kSliceNW);
  if (b < 0) return;
  const int64_t r = b * kSliceNW + wave_id();
  if (r >= a.n) return;
  const DistillRow o = distill_join(a, r);
  if (lane_id() == 0) distill_row_out(a, r, o);
}

// A vector's gradient from its logits v, ids t .. t + N - 1 of the set's row:
// off the list for all, then the listed ones one after the other, whose
// entries follow each other.
template <int N>
__device__ __forceinline__ void distill_grad_vec(const IdSet& on, const float* p, int t, float M, float M_off, float c,
                                                 float inv_s, float w_on, float f_off, float (&v)[N]) {
  uint32_t left = on.members<N>(t);
  float x[N];
#pragma unroll
  for (int l = 0; l < N; ++l) {
    x[l] = v[l];
    v[l] = __builtin_amdgcn_exp2f((v[l] - M_off) * c) * f_off;
  }
  if (left) {
    uint32_t e = on.entry(t);
    do {
      const uint32_t low = left & (0u - left);
      float y = x[0];
#pragma unroll
      for (int l = 1; l < N; ++l) y = low == 1u << l ? x[l] : y;
      const float d = (__builtin_amdgcn_exp2f((y - M) * c) * inv_s - p[e & (DSPARK_K_MAX - 1)]) * w_on;
#pragma unroll
      for (int l = 0; l < N; ++l) v[l] = low == 1u << l ? d : v[l];
      left ^= low;
      ++e;
    } while (left);
  }
}

// The gradient of one slice of one row; FROM_STATS: the row's numbers come
// from the forward call, otherwise they are joined here (and slice 0 writes
// the row's outputs).
template <int DT, bool FROM_STATS>
__global__ void __launch_bounds__(kSliceBS) distill_grad_kernel(DistillArgs a) {
  extern __shared__ uint32_t lds[];
  constexpr int N = kVec<DT>;
  __shared__ DistillRow sh;
  __shared__ float p[DSPARK_K_MAX];
  typedef typename El<DT>::T XT;
  int64_t r;
  int s;
  if (!row_slice(a.n, a.slices, r, s)) return;
  const int start = s * a.slice, V = a.V;
  const int size = V - start < a.slice ? V - start : a.slice;
  const int words = (a.slice + 31) / 32;
  const XT* x = static_cast<const XT*>(a.x) + r * a.x_stride;
  XT* g = static_cast<XT*>(a.grad) + r * a.grad_stride;
  IdSet on{lds, lds + words};
  if constexpr (FROM_STATS) {
    if (threadIdx.x == 0) {
      const double* st = a.stats_in + r * DSPARK_DISTILL_STATS;
      sh = DistillRow{a.status_in[r], st[0], st[1], st[2], st[3], st[4], 0.0};
    }
  } else if (wave_id() == 0) {
    const DistillRow o = distill_join(a, r);
    if (lane_id() == 0) {
      sh = o;
      if (s == 0) distill_row_out(a, r, o);
    }
  }
  on.clear(words);
  __syncthreads();
  int len = a.len[r];
  if (len < 0 || len > a.k_max) len = 0;
  if (sh.status != DSPARK_ST_OK || len == 0) {  // (uniform)
    float z[N];
#pragma unroll
    for (int l = 0; l < N; ++l) z[l] = 0.0f;
    for (int t = threadIdx.x * N; t < size; t += kSliceBS * N) store_vec<DT, N>(g, start + t, V, z);
    return;
  }
  const int32_t* ids = a.ids + r * a.k_max;
  const float* zl = a.logits + r * a.k_max;
  for (int e = threadIdx.x; e < len; e += kSliceBS) {
    const int32_t id = ids[e];
    const uint32_t t = (uint32_t)(id - start);
    if (id >= 0 && t < (uint32_t)size) {
      const int32_t prev = e > 0 ? ids[e - 1] : -1;
      on.add((int)t, prev < start ? -1 : prev - start, (uint32_t)e);
      p[e] = (float)exp((double)zl[e] * a.inv_t - sh.zm);
    }
  }
  __syncthreads();
  const float c = (float)(a.inv_t * (double)kLog2e);
  const float M = (float)sh.M, M_off = (float)sh.M_off, inv_s = (float)sh.inv_s;
  const double w = (double)a.weight[r] * a.inv_t;
  const float w_on = (float)w, f_off = (float)(sh.f_off * w);
  XT* const out = g + start;
  for_row<DT, true, kSliceBS>(x, start, size, [&](int t, float (&v)[N]) {
    distill_grad_vec<N>(on, p, t, M, M_off, c, inv_s, w_on, f_off, v);
    store_vec<DT, N>(out, t, size, v);
  });
}

// Loss and, with GRAD, gradient of one row by one workgroup, where the rows
// fill the chip or are short.  For the gradient the row is read again, out of
// the caches (the rows in work at once are about the last-level cache), so
// that HBM sees little more than one read and one write: 5,120 bf16 rows take
// 550 us, 4.8 TB/s of that read and write, where a copy reaches 5.2; in slices,
// which read HBM twice, 675.
template <int DT, int NWV, bool GRAD>
__global__ void __launch_bounds__(64 * NWV, NWV == 4 ? 6 : 8) distill_row_kernel(DistillArgs a) {
  constexpr int T = 64 * NWV, N = kVec<DT>, PER = DSPARK_K_MAX / T;
  extern __shared__ uint32_t lds[];
  __shared__ double sum_wave[NWV][4];
  __shared__ float m_wave[2][NWV], redf[NWV];
  __shared__ uint32_t redu[NWV];
  __shared__ float p[GRAD ? DSPARK_K_MAX : 1];
  __shared__ DistillRow sh;
  typedef typename El<DT>::T XT;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  const int V = a.V, tid = (int)threadIdx.x, words = (V + 31) / 32;
  const XT* x = static_cast<const XT*>(a.x) + r * a.x_stride;
  const int32_t* ids = a.ids + r * a.k_max;
  const float* zl = a.logits + r * a.k_max;
  const bool tail = a.lse != nullptr;
  const auto larger = [](float u, float v) { return __builtin_fmaxf(u, v); };
  const auto either = [](uint32_t u, uint32_t v) { return u | v; };
  constexpr float kNone = -__builtin_inff();

  int len = a.len[r];
  double w_list[PER];  // exp(z / T - zm) of this thread's list entries
  uint32_t wrong = 0;
  if (len < 0 || len > a.k_max) {
    wrong = 1u;
    len = 0;
  }
  if (len > 0 && tail && !finite_row_value(a.lse[r])) wrong |= 8u;
  IdSet on{lds, lds + words};
  on.clear(words);
  int32_t id[PER], prev[PER];
  float z[PER], zmax = kNone;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = j * T + tid;
    id[j] = prev[j] = -1;
    z[j] = kNone;
    if (e < len) {
      id[j] = ids[e];
      z[j] = zl[e];
      zmax = __builtin_fmaxf(zmax, z[j]);
      if (e > 0) prev[j] = ids[e - 1];
      if ((uint32_t)id[j] >= (uint32_t)V) wrong |= 2u;
      if (e > 0 && prev[j] >= id[j]) wrong |= 4u;
      if (!finite_row_value(z[j])) wrong |= 8u;
    }
  }
  wrong = group_reduce<NWV>(wrong, 0u, either, redu);  // (and the set is clear)
  int status = wrong ? DSPARK_ST_Q_BAD_LEN + (wrong & 1u ? 0 : wrong & 2u ? 1 : wrong & 4u ? 2 : 3) : DSPARK_ST_OK;
  const float c = (float)(a.inv_t * (double)kLog2e);
  if (status == DSPARK_ST_OK && len > 0) {  // (uniform)
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (id[j] >= 0) on.add(id[j], prev[j], (uint32_t)(j * T + tid));
    __syncthreads();
    // off the list: running maximum and sum, a vector moves the maximum at most once
    uint32_t flags = 0;
    float m = kNone, s_off = 0.0f;
    for_row<DT, false, T>(x, 0, V, [&](int t, float (&v)[N]) {
      const uint32_t bits = tail ? on.members<N>(t) : 0u;
      if (bits) {
#pragma unroll
        for (int l = 0; l < N; ++l) v[l] = (bits >> l) & 1u ? kNone : v[l];
      }
      float top = v[0];
#pragma unroll
      for (int l = 1; l < N; ++l) top = __builtin_fmaxf(top, v[l]);
      if (top > m) {
        s_off *= __builtin_amdgcn_exp2f((m - top) * c);  // (by 0 the first time)
        m = top;
      }
      const float ref = m == kNone ? 0.0f : m;
#pragma unroll
      for (int l = 0; l < N; ++l) s_off += __builtin_amdgcn_exp2f((v[l] - ref) * c);
    });
    if (s_off != s_off || m == __builtin_inff()) {  // a NaN or +inf: which, the logits tell
      for (int t = tid * N; t < V; t += T * N) {
        float v[N];
        load_vec<DT, N>(x, t, V, v);
#pragma unroll
        for (int l = 0; l < N; ++l) flags |= v[l] != v[l] ? 1u : v[l] == __builtin_inff() ? 2u : 0u;
      }
    }
    // the list's side, now that the row is in the caches
    const double zm = tail ? (double)a.lse[r] : (double)group_reduce<NWV>(zmax, kNone, larger, redf) * a.inv_t;
    double b0 = 0.0, b1 = 0.0;
    float m_own = kNone, s_on = 0.0f, x_list[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      x_list[j] = kNone;
      if (id[j] >= 0) {
        const float xj = x_list[j] = El<DT>::get(x, id[j]);
        m_own = __builtin_fmaxf(m_own, xj);
        if (tail) flags |= xj != xj ? 1u : xj == __builtin_inff() ? 2u : 0u;
      }
    }
    const double ref = m_own == kNone ? 0.0 : (double)m_own;  // (as in a slice)
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      w_list[j] = 0.0;
      if (id[j] >= 0) {
        const double lp = (double)z[j] * a.inv_t - zm;
        const double w = w_list[j] = exp(lp);
        if (w > 0.0) {
          b0 += w;
          b1 += w * (lp - ((double)x_list[j] - ref) * a.inv_t);
        }
      }
    }
    const float m_on = tail ? m_own : kNone;
    if (m_on > kNone) {
#pragma unroll
      for (int j = 0; j < PER; ++j) s_on += __builtin_amdgcn_exp2f((x_list[j] - m_on) * c);
    }
    // two meetings of the waves: the maxima, which all need, then the sums, which one wave joins
    m_wave[0][wave_id()] = wave_reduce(m, kNone, larger);
    m_wave[1][wave_id()] = wave_reduce(m_on, kNone, larger);
    __syncthreads();
    float M_off = kNone, M_on = kNone;
#pragma unroll
    for (int w = 0; w < NWV; ++w) {
      M_off = __builtin_fmaxf(M_off, m_wave[0][w]);
      M_on = __builtin_fmaxf(M_on, m_wave[1][w]);
    }
    if (b0 > 0.0) b1 += b0 * (((double)__builtin_fmaxf(M_off, M_on) - ref) * a.inv_t);
    const double f = m == kNone ? 0.0 : (double)__builtin_amdgcn_exp2f((m - M_off) * c);
    const double h = m_on == kNone ? 0.0 : (double)__builtin_amdgcn_exp2f((m_on - M_on) * c);
    const double w_off = wave_sum((double)s_off * f), w_on = wave_sum((double)s_on * h);
    b0 = wave_sum(b0);
    b1 = wave_sum(b1);
    flags = wave_reduce(flags, 0u, either);
    if (lane_id() == 0) {
      sum_wave[wave_id()][0] = w_off;
      sum_wave[wave_id()][1] = w_on;
      sum_wave[wave_id()][2] = b0;
      sum_wave[wave_id()][3] = b1;
      redu[wave_id()] = flags;
    }
    __syncthreads();
    if (wave_id() == 0) {
      const bool have = lane_id() < 4 * NWV;  // lane 4 w + i: sum i of wave w
      double v = have ? sum_wave[lane_id() >> 2][lane_id() & 3] : 0.0;
#pragma unroll
      for (int step = 4; step < 4 * NWV; step *= 2) v += __shfl_xor(v, step, 64);
      const double off = __shfl(v, 0, 64), sum_on = __shfl(v, 1, 64), t0 = __shfl(v, 2, 64), t1 = __shfl(v, 3, 64);
      flags = wave_reduce(lane_id() < NWV ? redu[lane_id()] : 0u, 0u, either);
      if (tid == 0) {
        DistillRow o{};
        o.status = distill_status(tail, t0, flags, __builtin_fmaxf(M_off, M_on));
        if (o.status == DSPARK_ST_OK) distill_finish(a.inv_t, tail, M_off, M_on, off, sum_on, t0, t1, zm, o);
        sh = o;
      }
    }
    __syncthreads();
    status = sh.status;
  }
  const bool live = status == DSPARK_ST_OK && len > 0;  // (uniform)
  if (tid == 0) {
    DistillRow o{};
    if (live) o = sh;
    o.status = status;
    distill_row_out(a, r, o);
  }
  if constexpr (!GRAD) return;
  XT* g = static_cast<XT*>(a.grad) + r * a.grad_stride;
  if (!live) {
    float v[N];
#pragma unroll
    for (int l = 0; l < N; ++l) v[l] = 0.0f;
    for (int t = tid * N; t < V; t += T * N) store_vec<DT, N>(g, t, V, v);
    return;
  }
  double norm = 1.0;  // the teacher's probabilities over w_list
  if (!tail) {
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < NWV; ++w) sum += sum_wave[w][2];
    norm = 1.0 / sum;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (id[j] >= 0) p[j * T + tid] = (float)(w_list[j] * norm);
  __syncthreads();
  const float M = (float)sh.M, M_off = (float)sh.M_off, inv_s = (float)sh.inv_s;
  const double w = (double)a.weight[r] * a.inv_t;
  const float w_on = (float)w, f_off = (float)(sh.f_off * w);
  for_row<DT, true, T>(x, 0, V, [&](int t, float (&v)[N]) {
    distill_grad_vec<N>(on, p, t, M, M_off, c, inv_s, w_on, f_off, v);
    store_vec<DT, N>(g, t, V, v);
  });
}

}  // namespace dspark
