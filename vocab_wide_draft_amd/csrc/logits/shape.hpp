// Shaping of logits: penalties for repeated tokens, biases, temperature and
// grammar masks (dspark_shape_logits).
//
// A workgroup owns one slice of the vocabulary of one request and all rows
// of the request there; a thread owns eight or sixteen of its tokens in every
// row.  The workgroup counts the request's tokens of its slice in LDS (bit 31: in the
// prompt; the other bits: times generated; integer additions, so the order
// does not matter) and lays the slice's biases beside them.  Each thread turns
// that into what a row needs of its tokens, in registers -- whether each was
// seen, and d = frequency c + presence [c > 0] - bias -- and streams its part
// of the rows through it: z = x m - d with m = 1 for an unseen token,
// 1 / repetition or repetition for a seen one, then z / T.  Both quotients
// are products with a reciprocal rounded once.  A drafted token changes its
// owner's registers between rows.  Every slice scans the whole history, so
// slices are not narrow (4,096 ids), and what is read from memory is asked
// for early: up to three rows ahead, the first rows and the first of the
// history before anything else.  6,144 bf16 rows with everything take 576 us
// (5.6 TB/s of what they read and write), their temperature alone 530.
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

// factors whose reciprocals keep all their bits
__device__ __forceinline__ bool in_range(float x) { return x >= 0x1p-100f && x <= 0x1p100f; }

// bit l of `bits` set: a, else b (the bit widened to a word that selects)
__device__ __forceinline__ float pick_bit(uint32_t bits, int l, float a, float b) {
  const uint32_t m = (uint32_t)((int32_t)(bits << (31 - l)) >> 31);
  return __uint_as_float((__float_as_uint(a) & m) | (__float_as_uint(b) & ~m));
}

// G: eights of logits per thread and row; kDepth: rows asked for ahead.
template <int TI, int TO, int NWV, int G, int kDepth>
__global__ void __launch_bounds__(64 * NWV) shape_kernel(ShapeArgs a) {
  constexpr int T = 64 * NWV, SLICE = 8 * G * T;
  constexpr int N = kVec<TO>, Q = 8 * G / N;  // Q vectors of N logits per thread and row
  static_assert(8 * (Q - 1) + N <= 32, "a word holds a bit for each of a thread's tokens");
  __shared__ __align__(16) uint32_t count[SLICE];
  __shared__ __align__(16) float bias[SLICE];
  __shared__ uint32_t bad;  // refusals of the whole request: bit code - BAD_HISTORY
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
  Raw<TI, N> ahead[kDepth][Q];
  uint32_t ahead_allowed[kDepth][Q];
  const auto fetch = [&](int i, Raw<TI, N> (&q)[Q]) {
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
  };
  const auto fetch_mask = [&](int64_t m, uint32_t (&allowed)[Q]) {
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
#pragma unroll
  for (int k = 0; k < kDepth; ++k)
    if (k < P) fetch(k, ahead[k]);

  // the first of the history (history_max of it may be read, whatever its length)
  constexpr int U = 32 / NWV;  // loads in flight per thread: 2,048 tokens of a workgroup
  const int32_t* hist = h.history + r * h.history_stride;
  int32_t token[U];
#pragma unroll
  for (int u = 0; u < U; ++u) token[u] = h.history && u * T + tid < h.history_max ? hist[u * T + tid] : 0;

  const float rep = h.repetition ? h.repetition[r] : 1.0f;
  const float freq = h.frequency ? h.frequency[r] : 0.0f;
  const float pres = h.presence ? h.presence[r] : 0.0f;
  const float temp = h.temperature ? h.temperature[r] : 1.0f;
  const float inv_rep = 1.0f / rep, inv_t = 1.0f / temp;
  const bool penal = rep != 1.0f || freq != 0.0f || pres != 0.0f;  // (uniform)
  const bool counted = penal && h.history;
  const bool drafted = penal && h.draft;
  const int64_t b0 = h.bias_offset ? h.bias_offset[r] : 0, b1 = h.bias_offset ? h.bias_offset[r + 1] : 0;

  uint32_t wrong = 0;
  if (!in_range(rep) || !in_range(temp) || !finite_f32(freq) || !finite_f32(pres))
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
  // the first of the biases and of the rows' masks, on their way while LDS is cleared
  int32_t bias_id = 0, bias_prev = -1;
  float bias_value = 0.0f;
  const auto fetch_bias = [&](int64_t e) {
    bias_id = h.bias_ids[e];
    bias_prev = e > b0 ? h.bias_ids[e - 1] : -1;
    bias_value = h.bias_values[e];
  };
  if (biased && b0 + tid < b1) fetch_bias(b0 + tid);
  int64_t ahead_mask[kDepth];
  int32_t ahead_draft[kDepth];
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    if (k < P) {
      ahead_mask[k] = mask_of(k);
      ahead_draft[k] = __builtin_amdgcn_readlane(lane_draft, k);
      fetch_mask(ahead_mask[k], ahead_allowed[k]);
    }
  }
  if (tid == 0) bad = 0u;
  const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) {
    if (counted || drafted) reinterpret_cast<float4*>(count)[i * T + tid] = none;
    if (biased) reinterpret_cast<float4*>(bias)[i * T + tid] = none;
  }
  __syncthreads();

  for (int i0 = tid; i0 < len; i0 += U * T) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * T;
      if (i < len) {
        if ((uint32_t)token[u] >= (uint32_t)V) wrong |= 1u;
        const uint32_t t = (uint32_t)(token[u] - start);
        if (t < (uint32_t)size) {
          if (i < plen) atomicOr(&count[t], kPrompt);
          else atomicAdd(&count[t], 1u);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = (int64_t)i0 + (U + u) * T;
      token[u] = i < len ? hist[i] : 0;
    }
  }
  if (biased) {
    for (int64_t e = b0 + tid; e < b1; e += T) {
      if (e != b0 + tid) fetch_bias(e);
      if ((uint32_t)bias_id >= (uint32_t)V || bias_prev >= bias_id || bias_value != bias_value || bias_value == __builtin_inff())
        wrong |= 1u << (DSPARK_ST_BAD_BIAS - DSPARK_ST_BAD_HISTORY);
      const uint32_t t = (uint32_t)(bias_id - start);
      if (t < (uint32_t)size) bias[t] = bias_value;  // (one entry per token in a list that is not refused)
    }
  }
  if (wrong) atomicOr(&bad, wrong);
  __syncthreads();
  wrong = bad;
  // this thread's tokens
  uint32_t seen = 0, hit = 0;  // bit 8 j + l: token l of vector j was seen; seen or biased
  float minus[Q][N];           // d
#pragma unroll
  for (int j = 0; j < Q; ++j) {
#pragma unroll
    for (int l = 0; l < N; l += 4) {
      const int t = (j * T + tid) * N + l;
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
      float4 f = none;
      if (counted || drafted) c = *reinterpret_cast<const uint4*>(count + t);
      if (biased) f = *reinterpret_cast<const float4*>(bias + t);
      const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
      const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t n = cs[i] & ~kPrompt;
        minus[j][l + i] = (n ? freq * (float)n + pres : 0.0f) - fs[i];
        seen |= cs[i] ? 1u << (8 * j + l + i) : 0u;
        hit |= cs[i] || fs[i] != 0.0f ? 1u << (8 * j + l + i) : 0u;
      }
    }
  }

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
      fetch(i + kDepth, ahead[k]);
      fetch_mask(ahead_mask[k], ahead_allowed[k]);
    }
    if (i > 0 && drafted) {
      if ((uint32_t)id >= (uint32_t)V) {
        wrong |= 1u;
      } else if ((uint32_t)(id - start) < (uint32_t)size) {
        const int t = id - start, l = t & (N - 1), v = t / N;  // (uniform)
        if (tid == v % T) {
          const int j = v / T;
          const uint32_t n = (count[t] += 1u) & ~kPrompt;
          const float d = (freq * (float)n + pres) - (biased ? bias[t] : 0.0f);
#pragma unroll
          for (int k = 0; k < Q * N; ++k)
            if (k == j * N + l) minus[k / N][k % N] = d;
          seen |= 1u << (8 * j + l);
          hit |= 1u << (8 * j + l);
        }
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
          if ((hit >> (8 * j)) & 0xffu) {
#pragma unroll
            for (int l = 0; l < N; ++l) {
              const float m = pick_bit(seen, 8 * j + l, z[j][l] > 0.0f ? inv_rep : rep, 1.0f);
              z[j][l] = __builtin_fmaf(z[j][l], m, -minus[j][l]);
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
