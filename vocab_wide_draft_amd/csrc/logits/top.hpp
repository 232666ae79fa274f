// The top logits of a row with the log-sum-exp of the whole row
// (dspark_top_logits).
//
// Rows of ordinary size are cut into slices of 8,192 ids, one workgroup each,
// which reads its slice once into registers.  A threshold that the k-th
// largest logit lies above with good odds comes from a sample of the row
// (2,048 logits, the same for every slice of the row), so that one pass
// yields the slice's maximum, its sum of exponentials and the few logits
// that may be among the top k.  A second kernel joins the slices of a row and
// selects exactly among those candidates.  A row whose candidates are too
// few or too many for their list (heavy ties, a sample that misleads) is
// selected from memory by that kernel's workgroup instead: slower, the same
// answer.
#pragma once
#include "../fast_q.hpp"
#include "../resident.hpp"
#include "slices.hpp"

namespace dspark {

struct TopArgs {
  int64_t n;
  const void* x;
  int64_t stride;
  int V;
  const int32_t* topk;
  int k_max;
  double inv_t;
  int32_t* ids;
  float* logits;
  int32_t* len;
  float* lse;
  int32_t* row_status;
};

// k of row r: -1 when out of range
__device__ __forceinline__ int row_k(const TopArgs& a, int64_t r) {
  const int cap = a.k_max < a.V ? a.k_max : a.V;
  const int k = a.topk ? a.topk[r] : cap;
  return k < 0 || k > cap ? -1 : k;
}

// writes the n entries of (sh.cid, sh.sx) and zeros behind them
__device__ __forceinline__ void write_top(const TopArgs& a, int64_t r, int n, const RowShared& sh) {
  for (int e = threadIdx.x; e < a.k_max; e += BS) {
    a.ids[r * a.k_max + e] = e < n ? (int32_t)sh.cid[e] : 0;
    a.logits[r * a.k_max + e] = e < n ? sh.sx[e] : 0.0f;
  }
}

__device__ __forceinline__ void finish_top(const TopArgs& a, int64_t r, int status, int n, float m, double sum) {
  if (threadIdx.x != 0) return;
  const bool ok = status == DSPARK_ST_OK;
  a.row_status[r] = status;
  a.len[r] = ok ? n : 0;
  if (a.lse) a.lse[r] = ok ? (float)((double)m * a.inv_t + log(sum)) : 0.0f;
}

// bf16 rows of up to NI * BS * 8 ids, held in registers
__global__ void __launch_bounds__(BS) top_bf16_kernel(TopArgs a) {
  __shared__ RowShared sh;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  Res R;
  res_load(R, static_cast<const uint16_t*>(a.x) + r * a.stride, a.V);
  const RStats st = res_stats(R, sh);
  const int k = row_k(a, r);
  int status = st.status;
  if (status == DSPARK_ST_OK && k < 0) status = DSPARK_ST_BAD_TOPK;
  int n = 0;
  double sum = 1.0;
  const float m = bf16_to_f32(st.m_raw);
  if (status == DSPARK_ST_OK) {
    if (a.lse) {
      const float c = (float)(a.inv_t * 1.4426950408889634);
      touch(R);
      double acc = 0.0;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4 v = fetch(R, i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          part += __builtin_amdgcn_exp2f((bf16_lo(w[j]) - m) * c);
          part += __builtin_amdgcn_exp2f((bf16_hi(w[j]) - m) * c);
        }
        acc += (double)part;
      }
      sum = block_sum<double>(acc, sh.bs);
    }
    if (k > 0) n = res_topk_support(R, st, k, sh);
  }
  __syncthreads();
  write_top(a, r, n, sh);
  finish_top(a, r, status, n, m, sum);
}

// a row streamed from memory
template <int DT>
__device__ __forceinline__ void top_stream_row(const TopArgs& a, int64_t r, RowShared& sh) {
  constexpr int ES = DT == DSPARK_BF16 ? 2 : 4;
  const Row<DT> row{static_cast<const char*>(a.x) + (size_t)r * (size_t)a.stride * ES, a.V};
  const Stats st = row_stats(row, sh.bs);
  const int k = row_k(a, r);
  int status = st.status;
  if (status == DSPARK_ST_OK && k < 0) status = DSPARK_ST_BAD_TOPK;
  int n = 0;
  double sum = 1.0;
  if (status == DSPARK_ST_OK) {
    const float c = (float)(a.inv_t * 1.4426950408889634);
    double acc = 0.0;
    uint32_t fin = 0;
    for_vecs<kPF, float, Row<DT>::EPV>(row.nvec(), [&](int q, float (&x)[Row<DT>::EPV]) { return row.load(q, x); },
                                       [&](int, const float (&x)[Row<DT>::EPV], int nv) {
      float part = 0.0f;
#pragma unroll
      for (int l = 0; l < Row<DT>::EPV; ++l) {
        part += __builtin_amdgcn_exp2f((x[l] - st.m) * c);  // (lanes past the end hold -inf)
        fin += l < nv && x[l] > -__builtin_inff() ? 1u : 0u;
      }
      acc += (double)part;
    });
    sum = block_sum<double>(acc, sh.bs);
    const uint32_t finite = block_sum<uint32_t>(fin, sh.bs);
    const int take = (uint32_t)k < finite ? k : (int)finite;  // -inf entries are not listed
    if (take > 0) n = stream_topk_support(row, st.m, st.tkey, take, sh);
  }
  __syncthreads();
  write_top(a, r, n, sh);
  finish_top(a, r, status, n, st.m, sum);
}

template <int DT>
__global__ void __launch_bounds__(BS) top_stream_kernel(TopArgs a) {
  __shared__ RowShared sh;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  top_stream_row<DT>(a, r, sh);
}

// ------------------------------------------------------- rows in slices
constexpr int kTopGroups = 4;                              // groups of eight logits per thread
constexpr int kTopSlice = kSliceStep * kTopGroups;         // ids of a slice
constexpr int kTopSlices = DSPARK_V_MAX / kTopSlice;       // slices of the longest row
constexpr int kTopSample = kSliceBS * 8;                   // logits sampled of a row: 64 runs of 32
constexpr int kTopPer = 8;                                 // candidates per thread of the selection, at most

struct TopPart {
  double sum;    // of exp((x - m) / T)
  float m, t;    // the slice's maximum; the row's threshold
  int32_t flags; // 1: a NaN, 2: a +inf
  int32_t count; // candidates (more than the list holds: too many)
};

// A candidate of a slice: its logit and its place in the slice.
template <int DT>
struct Cand;
template <>
struct Cand<DSPARK_BF16> {
  typedef uint32_t T;
  static __device__ __forceinline__ T make(float x, int t) { return (__float_as_uint(x) & 0xffff0000u) | (uint32_t)t; }
  static __device__ __forceinline__ float value(T c) { return __uint_as_float(c & 0xffff0000u); }
  static __device__ __forceinline__ int place(T c) { return (int)(c & 0xffffu); }
  static __device__ __forceinline__ uint32_t key(float x) { return key32(x) >> 16; }
};
template <>
struct Cand<DSPARK_F32> {
  typedef uint2 T;
  static __device__ __forceinline__ T make(float x, int t) { return make_uint2(__float_as_uint(x), (uint32_t)t); }
  static __device__ __forceinline__ float value(T c) { return __uint_as_float(c.x); }
  static __device__ __forceinline__ int place(T c) { return (int)c.y; }
  static __device__ __forceinline__ uint32_t key(float x) { return key32(x); }
};

struct TopSliceArgs {
  TopArgs a;
  int slices;
  int cap;      // candidates a slice's list holds
  int rank;     // the threshold is the rank-th largest of the sample's 256 maxima
  TopPart* part;  // [n][slices]
  void* cand;     // [n][slices][cap]
};

template <int DT>
__global__ void __launch_bounds__(kSliceBS) top_slice_kernel(TopSliceArgs q) {
  __shared__ __align__(16) float sample[kSliceBS];
  __shared__ float thr;
  __shared__ uint64_t scan[kSliceNW];
  __shared__ double red[kSliceNW];
  __shared__ float redf[kSliceNW];
  __shared__ uint32_t redu[kSliceNW];
  typedef typename El<DT>::T XT;
  const int64_t b = block_number(q.a.n * q.slices);
  if (b < 0) return;
  const int64_t r = b / q.slices;
  const int s = (int)(b - r * q.slices), start = s * kTopSlice, V = q.a.V, tid = (int)threadIdx.x;
  const XT* row = static_cast<const XT*>(q.a.x) + r * q.a.stride;
  const int step = (V / 64) & ~7;
  float smp[8], x[kTopGroups][8];
  load8<DT, false>(row, (tid >> 2) * step + (tid & 3) * 8, V, smp);
#pragma unroll
  for (int i = 0; i < kTopGroups; ++i) load8<DT, true>(row, start + (i * kSliceBS + tid) * 8, V, x[i]);
  float top = smp[0];
#pragma unroll
  for (int l = 1; l < 8; ++l) top = __builtin_fmaxf(top, smp[l]);
  if (top != top) top = -__builtin_inff();
  sample[tid] = top;
  if (tid == 0) thr = -__builtin_inff();
  __syncthreads();
  int above = 0;
  for (int u = 0; u < kSliceBS; u += 4) {
    const float4 o = *reinterpret_cast<const float4*>(sample + u);
    above += (o.x > top || (o.x == top && u < tid)) ? 1 : 0;
    above += (o.y > top || (o.y == top && u + 1 < tid)) ? 1 : 0;
    above += (o.z > top || (o.z == top && u + 2 < tid)) ? 1 : 0;
    above += (o.w > top || (o.w == top && u + 3 < tid)) ? 1 : 0;
  }
  if (above == q.rank - 1) thr = top;
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kTopGroups; ++i) {
#pragma unroll
    for (int l = 0; l < 8; ++l) m = __builtin_fmaxf(m, x[i][l]);
  }
  const float M = group_reduce<kSliceNW>(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); }, redf);
  const float t = thr, c = (float)(q.a.inv_t * 1.4426950408889634), ref = M == -__builtin_inff() ? 0.0f : M;
  float sum = 0.0f;
  uint32_t mask[kTopGroups];
  uint64_t counts = 0;  // four 16-bit fields
#pragma unroll
  for (int i = 0; i < kTopGroups; ++i) {
    mask[i] = 0u;
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      sum += __builtin_amdgcn_exp2f((x[i][l] - ref) * c);
      mask[i] |= x[i][l] >= t && x[i][l] > -__builtin_inff() ? 1u << l : 0u;
    }
    counts |= (uint64_t)__builtin_popcount(mask[i]) << (16 * i);
  }
  uint32_t flags = 0;
  if (sum != sum || m == __builtin_inff()) {
#pragma unroll
    for (int i = 0; i < kTopGroups; ++i) {
#pragma unroll
      for (int l = 0; l < 8; ++l) flags |= x[i][l] != x[i][l] ? 1u : x[i][l] == __builtin_inff() ? 2u : 0u;
    }
  }
  // places in the list: by group, then thread, then element -- id order
  const uint64_t inc = wave_incl_scan(counts);
  if (lane_id() == 63) scan[wave_id()] = inc;
  flags = group_reduce<kSliceNW>(flags, 0u, [](uint32_t u, uint32_t v) { return u | v; }, redu);
  const double total = group_reduce<kSliceNW>((double)sum, 0.0, [](double u, double v) { return u + v; }, red);
  uint64_t before = inc - counts, all = 0;
#pragma unroll
  for (int w = 0; w < kSliceNW; ++w) {
    if (w < wave_id()) before += scan[w];
    all += scan[w];
  }
  uint32_t base = 0;
  typename Cand<DT>::T* list = static_cast<typename Cand<DT>::T*>(q.cand) + (r * q.slices + s) * q.cap;
#pragma unroll
  for (int i = 0; i < kTopGroups; ++i) {
    uint32_t pos = base + ((uint32_t)(before >> (16 * i)) & 0xffffu);
    base += (uint32_t)(all >> (16 * i)) & 0xffffu;
    if (mask[i]) {
#pragma unroll
      for (int l = 0; l < 8; ++l) {
        if ((mask[i] >> l) & 1u) {
          if (pos < (uint32_t)q.cap) list[pos] = Cand<DT>::make(x[i][l], (i * kSliceBS + tid) * 8 + l);
          ++pos;
        }
      }
    }
  }
  if (tid == 0) {
    TopPart& p = q.part[r * q.slices + s];
    p.sum = total;
    p.m = M;
    p.t = t;
    p.flags = (int32_t)flags;
    p.count = (int32_t)base;
  }
}

// One workgroup per row: joins its slices and selects among the candidates.
template <int DT>
__global__ void __launch_bounds__(BS) top_select_kernel(TopSliceArgs q) {
  __shared__ RowShared sh;
  __shared__ uint32_t first[kTopSlices + 1];  // candidates before each slice
  __shared__ double row_sum;
  __shared__ float row_m;
  __shared__ int row_flags, row_over;
  const TopArgs& a = q.a;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  const TopPart* part = q.part + r * q.slices;
  if (threadIdx.x < 64) {  // two slices per lane
    const int l = lane_id();
    float m = -__builtin_inff(), mm[2] = {m, m};
    double ss[2] = {0.0, 0.0};
    uint32_t n[2] = {0u, 0u}, flags = 0u, over = 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (2 * l + j < q.slices) {
        const TopPart p = part[2 * l + j];
        mm[j] = p.m;
        ss[j] = p.sum;
        n[j] = (uint32_t)p.count;
        flags |= (uint32_t)p.flags;
        over |= p.count > q.cap ? 1u : 0u;
        m = __builtin_fmaxf(m, p.m);
      }
    }
    const float M = wave_reduce(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); });
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (mm[j] > -__builtin_inff()) sum += ss[j] * exp(((double)mm[j] - (double)M) * a.inv_t);
    sum = wave_sum(sum);
    flags = wave_reduce(flags, 0u, [](uint32_t u, uint32_t v) { return u | v; });
    over = wave_reduce(over, 0u, [](uint32_t u, uint32_t v) { return u | v; });
    const uint32_t inc = wave_incl_scan(n[0] + n[1]);
    first[2 * l] = inc - n[0] - n[1];
    first[2 * l + 1] = inc - n[1];
    if (l == 63) first[kTopSlices] = inc;
    if (l == 0) {
      row_sum = sum;
      row_m = M;
      row_flags = (int)flags;
      row_over = (int)over;
    }
  }
  __syncthreads();
  const uint32_t total = first[kTopSlices];
  const float M = row_m;
  const int k = row_k(a, r);
  int status = row_flags & 1 ? DSPARK_ST_ROW_NAN
               : row_flags & 2 ? DSPARK_ST_ROW_POSINF
               : M == -__builtin_inff() ? DSPARK_ST_ROW_ZERO_MASS
               : k < 0 ? DSPARK_ST_BAD_TOPK : DSPARK_ST_OK;
  int n = 0;
  if (status == DSPARK_ST_OK && k > 0) {
    if (row_over || total > (uint32_t)(kTopPer * BS) || (total < (uint32_t)k && part[0].t > -__builtin_inff())) {
      top_stream_row<DT>(a, r, sh);  // (uniform)
      return;
    }
    n = total < (uint32_t)k ? (int)total : k;
    // this thread's candidates, in id order
    const int per = (int)((total + BS - 1) / BS);
    float v[kTopPer];
    uint32_t id[kTopPer], key[kTopPer];
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {
      const uint32_t g = threadIdx.x * (uint32_t)per + (uint32_t)j;
      key[j] = 0u;  // (below every finite logit's key)
      v[j] = 0.0f;
      id[j] = 0u;
      if (j < per && g < total) {
        int lo = 0, hi = q.slices - 1;  // the last slice with first <= g
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (first[mid] <= g) lo = mid;
          else hi = mid - 1;
        }
        const typename Cand<DT>::T e = (static_cast<const typename Cand<DT>::T*>(q.cand) + (r * q.slices + lo) * q.cap)[g - first[lo]];
        v[j] = Cand<DT>::value(e);
        id[j] = (uint32_t)(lo * kTopSlice + Cand<DT>::place(e));
        key[j] = Cand<DT>::key(v[j]);
      }
    }
    // the n-th largest key: histograms of a range of keys, narrowed to one key or one full bin
    uint32_t hi = Cand<DT>::key(M), lo = 1u, T;
    if (part[0].t > -__builtin_inff()) lo = Cand<DT>::key(part[0].t);
    uint32_t need = (uint32_t)n, ties;  // of the keys equal to T, the first `ties` by id
    bool all_ge = false;
    for (;;) {
      const uint32_t range = hi - lo;
      const int shift = range < (uint32_t)kHistBins ? 0 : (32 - __builtin_clz(range)) - 12;
      const int nb = (int)(range >> shift) + 1;
      for (int i = threadIdx.x; i < nb; i += BS) sh.hist[i] = 0u;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kTopPer; ++j)
        if (key[j] >= lo && key[j] <= hi) atomicAdd(&sh.hist[(hi - key[j]) >> shift], 1u);
      __syncthreads();
      uint64_t above;
      const int bin = block_find_crossing(sh.hist, nb, need, true, sh, &above);
      need -= (uint32_t)above;
      const uint32_t in_bin = sh.hist[bin];
      __syncthreads();
      const uint32_t bhi = hi - ((uint32_t)bin << shift), width = (1u << shift) - 1u;
      const uint32_t blo = bhi - lo > width ? bhi - width : lo;
      if (in_bin == need || shift == 0) {
        all_ge = in_bin == need;
        T = all_ge ? blo : bhi;
        ties = need;
        break;
      }
      hi = bhi;
      lo = blo;
    }
    // places of the chosen ones: those above T (or all from T on), and the first ties, in id order
    uint32_t cnt = 0;  // low half: chosen for sure, high half: ties
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {
      if (all_ge ? key[j] >= T : key[j] > T) cnt += 1u;
      else if (!all_ge && key[j] == T) cnt += 0x10000u;
    }
    uint32_t pre = block_excl_scan<uint32_t>(cnt, sh.bs, nullptr);
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {
      const bool sure = all_ge ? key[j] >= T : key[j] > T, tie = !all_ge && key[j] == T;
      const uint32_t tb = pre >> 16;
      if (sure || (tie && tb < ties)) {
        const uint32_t pos = (pre & 0xffffu) + (tb < ties ? tb : ties);
        if (pos < (uint32_t)a.k_max) {
          a.ids[r * a.k_max + pos] = (int32_t)id[j];
          a.logits[r * a.k_max + pos] = v[j];
        }
      }
      pre += sure ? 1u : tie ? 0x10000u : 0u;
    }
  }
  for (int e = n + (int)threadIdx.x; e < a.k_max; e += BS) {
    a.ids[r * a.k_max + e] = 0;
    a.logits[r * a.k_max + e] = 0.0f;
  }
  finish_top(a, r, status, n, M, row_sum);
}

}  // namespace dspark
