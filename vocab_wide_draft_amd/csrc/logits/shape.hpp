// Shaping of logits: penalties for repeated tokens, biases, temperature and
// grammar masks (dspark_shape_logits).
//
// A workgroup owns one slice of the vocabulary of one request and all rows
// of the request there.  It counts the request's tokens of its slice in an
// LDS table (bit 31: in the prompt; the other bits: times generated; integer
// additions, so the order does not matter), then streams the slice of each
// row through the table, adding the drafted token between rows.
#pragma once
#include "slices.hpp"

namespace dspark {

struct ShapeArgs {
  const void* x;
  int64_t x_stride;
  void* out;
  int64_t out_stride;
  int32_t* row_status;
  int64_t n_requests;
  int V;
  int slices;  // per request
  int slice;   // ids of a slice (a multiple of kSliceStep)
  dspark_shaping how;
};

constexpr uint32_t kPrompt = 0x80000000u;

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

template <int TI, int TO>
__global__ void __launch_bounds__(kSliceBS) shape_kernel(ShapeArgs a) {
  extern __shared__ uint32_t lds[];
  __shared__ uint32_t bad;  // refusals of the whole request: bit code - BAD_HISTORY
  const int64_t b = block_number(a.n_requests * a.slices);
  if (b < 0) return;
  const int64_t r = b / a.slices;
  const int s = (int)(b - r * a.slices);
  const int start = s * a.slice, V = a.V;
  const int size = V - start < a.slice ? V - start : a.slice;  // ids of this slice
  const int words = (a.slice + 31) / 32;
  const dspark_shaping& h = a.how;
  uint32_t* const count = lds;
  const IdSet biased{lds + a.slice, lds + a.slice + words};

  const float rep = h.repetition ? h.repetition[r] : 1.0f;
  const float freq = h.frequency ? h.frequency[r] : 0.0f;
  const float pres = h.presence ? h.presence[r] : 0.0f;
  const float inv_t = 1.0f / (h.temperature ? h.temperature[r] : 1.0f);
  const bool penal = rep != 1.0f || freq != 0.0f || pres != 0.0f;  // (uniform)
  const bool counted = penal && h.history;
  const bool drafted = penal && h.draft;
  const int64_t b0 = h.bias_offset ? h.bias_offset[r] : 0, b1 = h.bias_offset ? h.bias_offset[r + 1] : 0;

  uint32_t wrong = 0;
  if (!(rep > 0.0f) || !finite_f32(rep) || !finite_f32(freq) || !finite_f32(pres) || !(inv_t > 0.0f) || !finite_f32(inv_t))
    wrong |= 1u << (DSPARK_ST_BAD_PENALTY - DSPARK_ST_BAD_HISTORY);
  const bool bias_ok = b0 >= 0 && b0 <= b1 && b1 <= h.bias_total;
  if (!bias_ok) wrong |= 1u << (DSPARK_ST_BAD_BIAS - DSPARK_ST_BAD_HISTORY);
  int64_t len = 0, plen = 0;
  if (counted) {
    len = h.history_len[r];
    plen = h.prompt_len ? h.prompt_len[r] : 0;
    if (len < 0 || len > h.history_max || plen < 0 || plen > len) {
      wrong |= 1u;
      len = 0;
    }
  }
  if (threadIdx.x == 0) bad = 0u;
  for (int i = threadIdx.x; i < a.slice; i += kSliceBS) count[i] = 0u;
  if (b1 > b0) IdSet(biased).clear(words);
  __syncthreads();

  if (counted) {
    const int32_t* hist = h.history + r * h.history_stride;
    for (int64_t i = threadIdx.x; i < len; i += kSliceBS) {
      const int32_t id = hist[i];
      if ((uint32_t)id >= (uint32_t)V) wrong |= 1u;
      const uint32_t t = (uint32_t)(id - start);
      if (t < (uint32_t)size) {
        if (i < plen) atomicOr(&count[t], kPrompt);
        else atomicAdd(&count[t], 1u);
      }
    }
  }
  if (bias_ok) {
    for (int64_t e = b0 + threadIdx.x; e < b1; e += kSliceBS) {
      const int32_t id = h.bias_ids[e], prev = e > b0 ? h.bias_ids[e - 1] : -1;
      const float v = h.bias_values[e];
      if ((uint32_t)id >= (uint32_t)V || prev >= id || v != v || v == __builtin_inff())
        wrong |= 1u << (DSPARK_ST_BAD_BIAS - DSPARK_ST_BAD_HISTORY);
      const uint32_t t = (uint32_t)(id - start);
      if (t < (uint32_t)size) IdSet(biased).add((int)t, prev < start ? -1 : prev - start, (uint32_t)(e - b0));
    }
  }
  if (wrong) atomicOr(&bad, wrong);
  __syncthreads();
  wrong = bad;

  typedef typename El<TI>::T XT;
  typedef typename El<TO>::T OT;
  constexpr int N = kVec<TO>;
  const int P = h.rows_per_request;
  const bool lookup = counted || drafted || b1 > b0;
  for (int i = 0; i < P; ++i) {
    const int64_t row = r * P + i;
    if (i > 0 && drafted) {
      const int32_t id = h.draft[r * h.draft_stride + i - 1];  // (uniform)
      if ((uint32_t)id >= (uint32_t)V) {
        wrong |= 1u;
      } else if ((uint32_t)(id - start) < (uint32_t)size) {
        __syncthreads();  // the row before has read the table
        if (threadIdx.x == 0) count[id - start] += 1u;
        __syncthreads();
      }
    }
    uint32_t now = wrong;
    const uint32_t* mask = nullptr;
    if (h.mask) {
      const int64_t m = h.mask_row ? h.mask_row[row] : row;
      if (m < -1 || m >= h.n_masks) now |= 1u << (DSPARK_ST_BAD_MASK - DSPARK_ST_BAD_HISTORY);
      else if (m >= 0) mask = h.mask + m * h.mask_stride;
    }
    const int status = now ? DSPARK_ST_BAD_HISTORY + __builtin_ctz(now) : DSPARK_ST_OK;
    if (s == 0 && threadIdx.x == 0) a.row_status[row] = status;
    const XT* x = static_cast<const XT*>(a.x) + row * a.x_stride;
    OT* o = static_cast<OT*>(a.out) + row * a.out_stride;
    for (int t = threadIdx.x * N; t < size; t += kSliceBS * N) {
      const int v = start + t;
      float z[N];
      if (status != DSPARK_ST_OK) {
#pragma unroll
        for (int l = 0; l < N; ++l) z[l] = -__builtin_inff();
        store_vec<TO, N>(o, v, V, z);
        continue;
      }
      load_vec<TI, N, true>(x, v, V, z);
      if (lookup) {
        uint32_t c[N];
        uint32_t any = 0;
        if (counted || drafted) {
#pragma unroll
          for (int l = 0; l < N; l += 4) {
            const uint4 q = *reinterpret_cast<const uint4*>(count + t + l);
            c[l] = q.x; c[l + 1] = q.y; c[l + 2] = q.z; c[l + 3] = q.w;
          }
#pragma unroll
          for (int l = 0; l < N; ++l) any |= c[l];
        }
        if (any) {
#pragma unroll
          for (int l = 0; l < N; ++l) {
            if (c[l]) {
              const uint32_t n = c[l] & ~kPrompt;
              float y = z[l] > 0.0f ? z[l] / rep : z[l] * rep;
              if (n) y = y - freq * (float)n - pres;
              z[l] = y;
            }
          }
        }
        const uint32_t bb = b1 > b0 ? biased.members<N>(t) : 0u;
        if (bb) {
#pragma unroll
          for (int l = 0; l < N; ++l)
            if ((bb >> l) & 1u) z[l] += h.bias_values[b0 + biased.entry(t + l)];
        }
      }
#pragma unroll
      for (int l = 0; l < N; ++l) z[l] *= inv_t;
      if (mask) {
        const uint32_t m = reinterpret_cast<const uint8_t*>(mask)[v >> 3] >> (v & 7);
#pragma unroll
        for (int l = 0; l < N; ++l) z[l] = (m >> l) & 1u ? z[l] : -__builtin_inff();
      }
      store_vec<TO, N>(o, v, V, z);
    }
  }
}

}  // namespace dspark
