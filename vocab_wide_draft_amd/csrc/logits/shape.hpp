// Shaping of logits: penalties for repeated tokens, biases, temperature and
// grammar masks (dspark_shape_logits).
//
// A workgroup owns one slice of the vocabulary of one request and all rows
// of the request there.  It counts the request's tokens of its slice in LDS
// (bit 31: in the prompt; the other bits: times generated; integer additions,
// so the order does not matter), turns the counts into what a row needs of a
// token -- whether it was seen, and d = frequency c + presence [c > 0] - bias
// -- and streams the slice of each row through that: z = x m - d with m = 1
// for an unseen token, 1 / repetition or repetition for a seen one, then
// z / T.  Both quotients are products with a reciprocal rounded once.  The
// drafted token is added between rows.  Every slice scans the whole history,
// so slices are wide (8,192 ids, 1,024 threads with eight logits of a row
// each) and a row's loads are issued a row ahead, the first before the
// history is read.
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
  dspark_shaping how;
};

constexpr uint32_t kPrompt = 0x80000000u;

__device__ __forceinline__ bool finite_f32(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// bit l of `bits` set: a, else b (the bit widened to a word that selects)
__device__ __forceinline__ float pick_bit(uint32_t bits, int l, float a, float b) {
  const uint32_t m = (uint32_t)((int32_t)(bits << (31 - l)) >> 31);
  return __uint_as_float((__float_as_uint(a) & m) | (__float_as_uint(b) & ~m));
}

template <int TI, int TO, int NWV>
__global__ void __launch_bounds__(64 * NWV, NWV == 16 ? 8 : 1) shape_kernel(ShapeArgs a) {
  constexpr int T = 64 * NWV, SLICE = 8 * T;
  constexpr int N = kVec<TO>, Q = 8 / N;  // Q vectors of N logits per thread and row
  __shared__ __align__(16) uint32_t count[SLICE];
  __shared__ __align__(16) float minus[SLICE];             // d of each token
  __shared__ __align__(16) uint8_t seen[SLICE / 8], hit[SLICE / 8];  // bits: seen; seen or biased
  __shared__ uint32_t bad;  // refusals of the whole request: bit code - BAD_HISTORY
  __shared__ float draft_bias;
  typedef typename El<TI>::T XT;
  typedef typename El<TO>::T OT;
  int64_t r;
  int s;
  if (!row_slice(a.n_requests, a.slices, r, s)) return;
  const int tid = (int)threadIdx.x, start = s * SLICE, V = a.V;
  const int size = V - start < SLICE ? V - start : SLICE;  // ids of this slice
  const dspark_shaping& h = a.how;
  const int P = h.rows_per_request;

  // what a row needs besides its logits, 64 rows at a time, one per lane: its
  // mask (-1: none) and the token drafted before it
  int32_t lane_mask = -1, lane_draft = 0;
  const auto fetch_lanes = [&](int i) {
    const int k = i + lane_id();
    if (h.mask && k < P) lane_mask = h.mask_row ? h.mask_row[r * P + k] : 0;
    if (h.draft && k > 0 && k < P) lane_draft = h.draft[r * h.draft_stride + k - 1];
  };
  fetch_lanes(0);
  // a row's logits and mask bits of this thread, kDepth rows ahead of their use
  constexpr int kDepth = TI == DSPARK_F32 ? 2 : 3;
  Raw<TI, N> ahead[kDepth][Q];
  uint32_t ahead_allowed[kDepth][Q];
  const auto fetch = [&](int i, int64_t m, Raw<TI, N> (&q)[Q], uint32_t (&allowed)[Q]) {
    const XT* x = static_cast<const XT*>(a.x) + (r * P + i) * a.x_stride + start;
    if (size == SLICE) {  // (uniform)
#pragma unroll
      for (int j = 0; j < Q; ++j) q[j] = raw_whole<TI, N, true>(x, (uint32_t)(j * T + tid) * N);
    } else {
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const int t = (j * T + tid) * N;
        if (t < size) q[j] = raw_vec<TI, N, true>(x, t, size);
      }
    }
#pragma unroll
    for (int j = 0; j < Q; ++j) allowed[j] = 0xffu;
    if (m >= 0 && m < h.n_masks) {
      const uint8_t* mask = reinterpret_cast<const uint8_t*>(h.mask + m * h.mask_stride) + (start >> 3);
#pragma unroll
      for (int j = 0; j < Q; ++j) {
        const uint32_t t = (uint32_t)(j * T + tid) * N;
        if (t < (uint32_t)size) allowed[j] = (uint32_t)mask[t >> 3];
      }
    }
  };
  // the mask of row i, which fetch_lanes has read
  const auto mask_of = [&](int i) -> int64_t {
    if (!h.mask) return -1;
    if (!h.mask_row) return r * P + i;
    return __builtin_amdgcn_readlane(lane_mask, i & 63);
  };
  int64_t ahead_mask[kDepth];
  int32_t ahead_draft[kDepth];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k < P) {
      ahead_mask[k] = mask_of(k);
      ahead_draft[k] = __builtin_amdgcn_readlane(lane_draft, k);
      fetch(k, ahead_mask[k], ahead[k], ahead_allowed[k]);
    }
  }

  const float rep = h.repetition ? h.repetition[r] : 1.0f;
  const float freq = h.frequency ? h.frequency[r] : 0.0f;
  const float pres = h.presence ? h.presence[r] : 0.0f;
  const float inv_rep = 1.0f / rep, inv_t = 1.0f / (h.temperature ? h.temperature[r] : 1.0f);
  const bool penal = rep != 1.0f || freq != 0.0f || pres != 0.0f;  // (uniform)
  const bool counted = penal && h.history;
  const bool drafted = penal && h.draft;
  const int64_t b0 = h.bias_offset ? h.bias_offset[r] : 0, b1 = h.bias_offset ? h.bias_offset[r + 1] : 0;

  uint32_t wrong = 0;
  if (!(rep > 0.0f) || !finite_f32(rep) || !finite_f32(freq) || !finite_f32(pres) || !(inv_t > 0.0f) || !finite_f32(inv_t))
    wrong |= 1u << (DSPARK_ST_BAD_PENALTY - DSPARK_ST_BAD_HISTORY);
  const bool bias_ok = b0 >= 0 && b0 <= b1 && b1 <= h.bias_total;
  if (!bias_ok) wrong |= 1u << (DSPARK_ST_BAD_BIAS - DSPARK_ST_BAD_HISTORY);
  int len = 0, plen = 0;
  if (counted) {
    len = h.history_len[r];
    plen = h.prompt_len ? h.prompt_len[r] : 0;
    if (len < 0 || len > h.history_max || plen < 0 || plen > len) {
      wrong |= 1u;
      len = 0;
    }
  }
  const bool biased = bias_ok && b1 > b0;
  const bool changed = counted || drafted || biased;
  if (tid == 0) bad = 0u;
  if (changed) {
#pragma unroll
    for (int i = 0; i < 2; ++i) reinterpret_cast<uint4*>(count)[i * T + tid] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();

  if (counted) {
    const int32_t* hist = h.history + r * h.history_stride;
    constexpr int U = 4;  // loads in flight
    for (int i0 = tid; i0 < len; i0 += U * T) {
      int32_t id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) id[u] = i0 + u * T < len ? hist[i0 + u * T] : start;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * T;
        if (i < len) {
          if ((uint32_t)id[u] >= (uint32_t)V) wrong |= 1u;
          const uint32_t t = (uint32_t)(id[u] - start);
          if (t < (uint32_t)size) {
            if (i < plen) atomicOr(&count[t], kPrompt);
            else atomicAdd(&count[t], 1u);
          }
        }
      }
    }
  }
  if (changed) {  // this thread's eight tokens: from counts to what a row needs
    __syncthreads();
    uint32_t c[8], bits = 0;
    float d[8];
#pragma unroll
    for (int l = 0; l < 8; l += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(count + tid * 8 + l);
      c[l] = q.x; c[l + 1] = q.y; c[l + 2] = q.z; c[l + 3] = q.w;
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const uint32_t n = c[l] & ~kPrompt;
      d[l] = n ? freq * (float)n + pres : 0.0f;
      bits |= c[l] ? 1u << l : 0u;
    }
#pragma unroll
    for (int l = 0; l < 8; l += 4) *reinterpret_cast<float4*>(minus + tid * 8 + l) = make_float4(d[l], d[l + 1], d[l + 2], d[l + 3]);
    seen[tid] = hit[tid] = (uint8_t)bits;
    __syncthreads();
  }
  if (biased) {
    for (int64_t e = b0 + tid; e < b1; e += T) {
      const int32_t id = h.bias_ids[e], prev = e > b0 ? h.bias_ids[e - 1] : -1;
      const float v = h.bias_values[e];
      if ((uint32_t)id >= (uint32_t)V || prev >= id || v != v || v == __builtin_inff())
        wrong |= 1u << (DSPARK_ST_BAD_BIAS - DSPARK_ST_BAD_HISTORY);
      const uint32_t t = (uint32_t)(id - start);
      if (t < (uint32_t)size) {  // (one entry per token in a list that is not refused)
        minus[t] -= v;
        atomicOr(reinterpret_cast<uint32_t*>(hit) + (t >> 5), 1u << (t & 31));
      }
    }
  }
  if (wrong) atomicOr(&bad, wrong);
  __syncthreads();
  wrong = bad;

  for (int i0 = 0; i0 < P; i0 += kDepth) {
#pragma unroll
    for (int k = 0; k < kDepth; ++k) {
    const int i = i0 + k;
    if (i >= P) break;
    const int64_t row = r * P + i;
    float z[Q][N];
    uint32_t allowed[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      unpack<TI, N>(ahead[k][j], z[j]);
      allowed[j] = ahead_allowed[k][j] >> ((j * T + tid) * N & 7);
    }
    const int64_t m = ahead_mask[k];
    const int32_t id = ahead_draft[k];  // drafted before this row (uniform)
    if (i + kDepth < P) {
      if (((i + kDepth) & 63) == 0) fetch_lanes(i + kDepth);
      ahead_mask[k] = mask_of(i + kDepth);
      ahead_draft[k] = __builtin_amdgcn_readlane(lane_draft, (i + kDepth) & 63);
      fetch(i + kDepth, ahead_mask[k], ahead[k], ahead_allowed[k]);
    }
    if (i > 0 && drafted) {
      if ((uint32_t)id >= (uint32_t)V) {
        wrong |= 1u;
      } else if ((uint32_t)(id - start) < (uint32_t)size) {
        const int t = id - start;
        if (tid == 0) draft_bias = 0.0f;
        __syncthreads();  // the row before has read the table
        if (biased) {
          for (int64_t e = b0 + tid; e < b1; e += T)
            if (h.bias_ids[e] == id) draft_bias = h.bias_values[e];
          __syncthreads();
        }
        if (tid == 0) {
          const uint32_t n = (count[t] += 1u) & ~kPrompt;
          minus[t] = (freq * (float)n + pres) - draft_bias;
          seen[t >> 3] |= (uint8_t)(1u << (t & 7));
          hit[t >> 3] |= (uint8_t)(1u << (t & 7));
        }
        __syncthreads();
      }
    }
    uint32_t now = wrong;
    if (m < -1 || m >= h.n_masks) now |= 1u << (DSPARK_ST_BAD_MASK - DSPARK_ST_BAD_HISTORY);
    const int status = now ? DSPARK_ST_BAD_HISTORY + __builtin_ctz(now) : DSPARK_ST_OK;
    if (s == 0 && tid == 0) a.row_status[row] = status;
    OT* o = static_cast<OT*>(a.out) + row * a.out_stride + start;
#pragma unroll
    for (int j = 0; j < Q; ++j) {
      const int t = (j * T + tid) * N;
      if (t < size) {
        if (status != DSPARK_ST_OK) {
          allowed[j] = 0u;
        } else {
          if (changed && ((uint32_t)hit[t >> 3] >> (t & 7) & ((1u << N) - 1u))) {
            const uint32_t sb = (uint32_t)seen[t >> 3] >> (t & 7);
            float d[N];
#pragma unroll
            for (int l = 0; l < N; l += 4) {
              const float4 q = *reinterpret_cast<const float4*>(minus + t + l);
              d[l] = q.x; d[l + 1] = q.y; d[l + 2] = q.z; d[l + 3] = q.w;
            }
#pragma unroll
            for (int l = 0; l < N; ++l) {
              const float m = pick_bit(sb, l, z[j][l] > 0.0f ? inv_rep : rep, 1.0f);
              z[j][l] = __builtin_fmaf(z[j][l], m, -d[l]);
            }
          }
#pragma unroll
          for (int l = 0; l < N; ++l) z[j][l] *= inv_t;
        }
        if (h.mask || status != DSPARK_ST_OK) {
#pragma unroll
          for (int l = 0; l < N; ++l) z[j][l] = pick_bit(allowed[j], l, z[j][l], -__builtin_inff());
        }
        store_vec<TO, N>(o, t, size, z[j]);
      }
    }
    }
  }
}

}  // namespace dspark
