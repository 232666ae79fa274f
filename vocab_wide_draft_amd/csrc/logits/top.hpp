// The top logits of a row with the log-sum-exp of the whole row
// (dspark_top_logits).
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

// rows streamed from memory
template <int DT>
__global__ void __launch_bounds__(BS) top_stream_kernel(TopArgs a) {
  __shared__ RowShared sh;
  constexpr int ES = DT == DSPARK_BF16 ? 2 : 4;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
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

}  // namespace dspark
