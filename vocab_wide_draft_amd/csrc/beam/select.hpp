// Beam search's selection over beams and vocabulary (dspark_beam_select).
//
// Rows are cut into slices, one workgroup each, which reads its slice once
// into registers: its maxima and sums of exponentials (a reference for each
// wave), and the logits that may be among the row's best.  A second kernel
// joins a request: each of its waves takes beams, joins their slices into the
// log-sum-exp and the sorted list of the beam's best, and one wave merges the
// beams' lists, a beam to a lane.
//
// Order.  Within a beam the order of scores is the order of logits, and the
// lists are exact whatever the log-sum-exp.  Between beams it hangs on their
// log-sum-exps, which binary32 exponentials give to kLseOff at most (an
// exponent t is rounded by |t| 2^-24 in base 2, the hardware exponential by
// 2^-23, eight terms are added in binary32 before binary64 takes them: with
// the weights' mean |t| below 18 for 2^20 logits, 2^-24 (0.7 * 18 + 2 + 8) =
// 1.4e-6).  Where two neighbours in the merged order of different beams lie
// closer than twice that, their beams' log-sum-exps are computed again in
// binary64, and the lists are merged again.
#pragma once
#include "../logits/slices.hpp"
#include "../logits/top.hpp"

namespace dspark {

constexpr int kBeams = 64;      // beams of a request: a lane each
constexpr int kBeamOut = 128;   // candidates selected
constexpr double kLseOff = 2e-6;

struct BeamPart {
  float m[kSliceNW], sum[kSliceNW];  // of each wave: its maximum, the sum of exponentials relative to it
  int32_t flags;                     // 1: a NaN, 2: a +inf
  int32_t count;                     // candidates in the slice's list
};

struct BeamArgs {
  TopArgs x;  // rows, their width, temperature 1
  const float* scores;
  const int32_t* finished;
  int beams, n_out, end_token;
  int64_t requests;
  int32_t *parent, *token, *out_finished, *len, *status;
  float* score;
  int slices, cap;  // of a row; candidates of a slice's list
  BeamPart* part;   // [rows][slices]
  uint64_t* cand;   // [rows][slices][cap]
};

// whether a beam takes part with its row
__device__ __forceinline__ bool beam_live(const BeamArgs& a, int64_t row) {
  const float s = a.scores[row];
  return __builtin_fabsf(s) < __builtin_inff() && !(a.finished && a.finished[row] != 0);
}

// A candidate: its logit's order key above its id's complement, so that the
// larger one comes first (the larger logit, then the lower id), no two are
// alike and none is 0.
__device__ __forceinline__ uint64_t beam_key(float x, int id) { return ((uint64_t)key32(x) << 32) | (uint32_t)~id; }
__device__ __forceinline__ int beam_id(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float beam_logit(uint64_t k) { return top_key_value<DSPARK_F32>((uint32_t)(k >> 32)); }

template <int DT, int U>
__global__ void __launch_bounds__(kSliceBS) beam_slice_kernel(BeamArgs a) {
  constexpr int N = kVec<DT>, SLICE = U * kSliceBS * N;
  __shared__ __align__(16) uint32_t most[kSliceBS];
  __shared__ float thr;
  __shared__ uint32_t any_flags, held, counts[kSliceNW];
  typedef typename El<DT>::T XT;
  int64_t r;
  int s;
  if (!row_slice(a.x.n, a.slices, r, s)) return;
  BeamPart& p = a.part[r * a.slices + s];
  const int start = s * SLICE, V = a.x.V, tid = (int)threadIdx.x;
  if (!beam_live(a, r)) return;  // (uniform; the join does not read its record)
  const XT* row = static_cast<const XT*>(a.x.x) + r * a.x.stride;
  Raw<DT, N> raw[U];
  if (start + SLICE <= V) {  // (uniform)
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = raw_whole<DT, N, true>(row + start, (uint32_t)(i * kSliceBS + tid) * N);
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = raw_vec<DT, N, true>(row + start, (i * kSliceBS + tid) * N, V - start);
  }
  if (tid == 0) {
    any_flags = 0u;
    held = 0u;
  }
  float x[U][N];
#pragma unroll
  for (int i = 0; i < U; ++i) unpack<DT, N>(raw[i], x[i]);
  float m = x[0][0];
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) m = __builtin_fmaxf(m, x[i][l]);
  }
  most[tid] = m != m || m == -__builtin_inff() ? 0u : key32(m) >> 16;
  __syncthreads();
  if (wave_id() == 0) {
    // the largest 16-bit key that at least n_out of the threads' maxima reach: n_out logits of the slice do, too
    const uint4 o = *reinterpret_cast<const uint4*>(most + 4 * lane_id());
    uint32_t T = 0;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t up = T | (1u << bit);
      const int reach = __builtin_popcountll(__ballot(o.x >= up)) + __builtin_popcountll(__ballot(o.y >= up)) +
                        __builtin_popcountll(__ballot(o.z >= up)) + __builtin_popcountll(__ballot(o.w >= up));
      if (reach >= a.n_out) T = up;
    }
    const float t = top_key_value<DSPARK_BF16>(T);  // (-inf is no candidate)
    if (lane_id() == 0) thr = t >= -3.4028235e38f ? t : -3.4028235e38f;
  }
  const float M = wave_reduce(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); });
  const float ref = M == -__builtin_inff() ? 0.0f : M;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < U; ++i) sum += (double)exp_sum(a.x, ref, x[i]);
  if (sum != sum || M == __builtin_inff()) {  // a NaN or a +inf in this thread, or the wave's
    uint32_t flags = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int l = 0; l < N; ++l) flags |= x[i][l] != x[i][l] ? 1u : x[i][l] == __builtin_inff() ? 2u : 0u;
    }
    if (flags) atomicOr(&any_flags, flags);
  }
  const double wsum = wave_sum(sum);
  if (lane_id() == 63) {
    p.m[wave_id()] = M;
    p.sum[wave_id()] = (float)wsum;
  }
  __syncthreads();
  const float t = thr;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) mine += x[i][l] >= t ? 1u : 0u;
  }
  const uint32_t of_wave = wave_sum(mine);
  if (lane_id() == 0) counts[wave_id()] = of_wave;
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int w = 0; w < kSliceNW; ++w) total += counts[w];
  uint64_t least = (uint64_t)key32(t) << 32;
  if (total > (uint32_t)a.cap) {
    // too many (equal logits): the key that exactly n_out of them reach, by
    // halving (uniform; a sum over the workgroup each time)
    uint64_t lo = least, hi = ~0ull;  // reached by more than n_out, by fewer
    for (;;) {
      const uint64_t mid = lo + ((hi - lo) >> 1);
      mine = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) {
#pragma unroll
        for (int l = 0; l < N; ++l)
          mine += x[i][l] >= t && beam_key(x[i][l], start + (i * kSliceBS + tid) * N + l) >= mid ? 1u : 0u;
      }
      const uint32_t w = wave_sum(mine);
      __syncthreads();
      if (lane_id() == 0) counts[wave_id()] = w;
      __syncthreads();
      total = 0;
#pragma unroll
      for (int v = 0; v < kSliceNW; ++v) total += counts[v];
      least = mid;
      if (total == (uint32_t)a.n_out || hi - lo <= 1) break;  // (no two keys are alike: the former comes)
      if (total > (uint32_t)a.n_out) lo = mid;
      else hi = mid;
    }
  }
  uint64_t* list = a.cand + (r * a.slices + s) * a.cap;
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) {
      if (x[i][l] >= t) {
        const uint64_t k = beam_key(x[i][l], start + (i * kSliceBS + tid) * N + l);
        if (k >= least) {
          const uint32_t at = atomicAdd(&held, 1u);  // in any order: the keys have one
          if (at < (uint32_t)a.cap) list[at] = k;
        }
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.flags = (int32_t)any_flags;
    p.count = held < (uint32_t)a.cap ? (int)held : a.cap;
  }
}

// what lanes of a wave wrote to LDS is there for the others
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

constexpr int kBeamPer = 16;       // candidates of a lane in the join
constexpr int kBeamSlices = 128;   // slices of a row: two to a lane

// The n largest of the wave's keys (0: none; no two alike), or all of them:
// the least key that is among them.
template <int PER>
__device__ __forceinline__ uint64_t beam_cut(const uint64_t (&key)[PER], int n, int* found) {
  uint64_t top = 0, low = ~0ull;
  int all = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    top = key[j] > top ? key[j] : top;
    low = key[j] && key[j] < low ? key[j] : low;
    all += __builtin_popcountll(__ballot(key[j] != 0));
  }
  if (all <= n) {
    *found = all;
    return 1ull;
  }
  *found = n;
  uint64_t hi = wave_reduce(top, (uint64_t)0, [](uint64_t u, uint64_t v) { return u > v ? u : v; });
  uint64_t lo = wave_reduce(low, ~(uint64_t)0, [](uint64_t u, uint64_t v) { return u < v ? u : v; });
  for (;;) {  // reached by more than n: lo; by fewer: past hi
    const uint64_t mid = lo + ((hi - lo) >> 1) + 1;
    int reach = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) reach += __builtin_popcountll(__ballot(key[j] >= mid));
    if (reach == n || hi - lo <= 1) return mid;  // (no two keys are alike: the former comes)
    if (reach > n) lo = mid;
    else hi = mid - 1;
  }
}

// binary64 log-sum-exp of a row by the whole workgroup (every thread calls
// and gets it)
template <int DT, int NWV>
__device__ double beam_exact_lse(const BeamArgs& a, int64_t r, float M, double* scratch) {
  constexpr int N = kVec<DT>;
  const typename El<DT>::T* row = static_cast<const typename El<DT>::T*>(a.x.x) + r * a.x.stride;
  double sum = 0.0;
  for (int v = (int)threadIdx.x * N; v < a.x.V; v += NWV * 64 * N) {
    float x[N];
    load_vec<DT, N>(row, v, a.x.V, x);
#pragma unroll
    for (int l = 0; l < N; ++l) sum += exp((double)x[l] - (double)M);
  }
  sum = group_reduce<NWV>(sum, 0.0, [](double u, double v) { return u + v; }, scratch);
  return (double)M + log(sum);
}

// One workgroup per request.
template <int DT, int NWV>
__global__ void __launch_bounds__(64 * NWV) beam_join_kernel(BeamArgs a) {
  extern __shared__ __align__(16) uint64_t lists[];  // [beams][n_out], sorted
  __shared__ uint32_t first[NWV][kBeamSlices + 1];
  __shared__ uint64_t kept[NWV][kBeamOut];
  __shared__ double lse[kBeams], scratch[NWV];
  __shared__ float row_m[kBeams];
  __shared__ int32_t n_list[kBeams], flags[kBeams];
  __shared__ uint64_t again;
  const int64_t q = block_number(a.requests);
  if (q < 0) return;
  const int lane = lane_id(), wave = wave_id(), n = a.n_out;
  for (int b = wave; b < a.beams; b += NWV) {  // (uniform in the wave)
    const int64_t r = q * a.beams + b;
    const float s = a.scores[r];
    const bool ended = a.finished && a.finished[r] != 0;
    if (!beam_live(a, r)) {
      if (lane == 0) {
        const bool bad = s != s || s == __builtin_inff();
        flags[b] = bad ? 4 : 0;
        n_list[b] = ended && !bad && s > -__builtin_inff() ? 1 : 0;
        lists[b * n] = beam_key(0.0f, a.end_token);  // a score of its own: s + 0 - 0
        lse[b] = 0.0;
        row_m[b] = 0.0f;
      }
      continue;
    }
    const BeamPart* part = a.part + r * a.slices;
    // the slices' lists and sums: two slices to a lane
    constexpr float kNone = -__builtin_inff();
    uint32_t c[2] = {0u, 0u}, f = 0u;
    float m[2][kSliceNW], sum[2][kSliceNW], mine = kNone;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int w = 0; w < kSliceNW; ++w) {
        m[j][w] = kNone;
        sum[j][w] = 0.0f;
      }
      if (2 * lane + j < a.slices) {
        const BeamPart& p = part[2 * lane + j];
        c[j] = (uint32_t)p.count;
        f |= (uint32_t)p.flags;
#pragma unroll
        for (int w = 0; w < kSliceNW; ++w) {
          m[j][w] = p.m[w];
          sum[j][w] = p.sum[w];
          mine = __builtin_fmaxf(mine, m[j][w]);
        }
      }
    }
    f = wave_reduce(f, 0u, [](uint32_t u, uint32_t v) { return u | v; });
    const float M = wave_reduce(mine, kNone, [](float u, float v) { return __builtin_fmaxf(u, v); });
    const uint32_t inc = wave_incl_scan(c[0] + c[1]);
    first[wave][2 * lane] = inc - c[0] - c[1];
    first[wave][2 * lane + 1] = inc - c[1];
    if (lane == 63) first[wave][kBeamSlices] = inc;
    double total = 0.0, at = 0.0;
    if (!f && M > kNone) {  // (uniform)
      const double top = sum_reference(a.x, M);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int w = 0; w < kSliceNW; ++w)
          if (m[j][w] > kNone) total += (double)sum[j][w] * exp(sum_reference(a.x, m[j][w]) - top);
      }
      total = wave_sum(total);
      at = top + log(total);
    }
    wave_sync();
    const int count = f || !(M > kNone) ? 0 : (int)first[wave][kBeamSlices];
    int held = 0;
    for (int g0 = 0; g0 < count; g0 += (kBeamPer - 2) * 64) {
      uint64_t key[kBeamPer];
#pragma unroll
      for (int j = 0; j < 2; ++j) key[j] = j * 64 + lane < held ? kept[wave][j * 64 + lane] : 0ull;  // the best so far
#pragma unroll
      for (int j = 2; j < kBeamPer; ++j) {
        const int g = g0 + (j - 2) * 64 + lane;
        key[j] = 0ull;
        if (g < count) {
          int lo = 0, hi = a.slices - 1;  // the last slice that starts at or before g
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[wave][mid] <= (uint32_t)g) lo = mid;
            else hi = mid - 1;
          }
          key[j] = a.cand[(r * a.slices + lo) * a.cap + g - first[wave][lo]];
        }
      }
      const uint64_t least = beam_cut(key, n, &held);
      int before = 0;
      wave_sync();
#pragma unroll
      for (int j = 0; j < kBeamPer; ++j) {
        const uint64_t in = __ballot(key[j] >= least);
        if (key[j] >= least) kept[wave][before + __builtin_popcountll(in & ((1ull << lane) - 1ull))] = key[j];
        before += __builtin_popcountll(in);
      }
      wave_sync();
    }
    // sorted: an entry's place is the number of larger ones
#pragma unroll
    for (int j = 0; j < kBeamOut / 64; ++j) {
      const int e = j * 64 + lane;
      if (j * 64 < held) {  // (uniform)
        const uint64_t own = e < held ? kept[wave][e] : 0ull;
        int larger = 0;
        for (int i = 0; i < held; ++i) larger += kept[wave][i] > own ? 1 : 0;
        if (e < held) lists[b * n + larger] = own;
      }
    }
    if (lane == 0) {
      flags[b] = (int)f;
      n_list[b] = held;
      lse[b] = at;
      row_m[b] = M;
    }
  }
  if (threadIdx.x == 0) again = 0ull;
  __syncthreads();

  // the merge: a beam to a lane of the first wave
  const int64_t at_out = q * n;
  const bool here = lane < a.beams;
  const float s = here ? a.scores[q * a.beams + lane] : 0.0f;
  const bool ended = here && a.finished && a.finished[q * a.beams + lane] != 0;
  const uint32_t bad = wave_reduce(here ? (uint32_t)flags[lane] : 0u, 0u, [](uint32_t u, uint32_t v) { return u | v; });
  const int status = bad & 1u ? DSPARK_ST_ROW_NAN : bad & 2u ? DSPARK_ST_ROW_POSINF : bad & 4u ? DSPARK_ST_BAD_SCORE : DSPARK_ST_OK;
  const auto merge = [&]() {  // by the first wave; the beams whose order is not certain
    constexpr double kNone = -__builtin_inf();
    const int mine = here && status == DSPARK_ST_OK ? n_list[lane] : 0;
    const double base = here ? (double)s : 0.0, minus = here ? lse[lane] : 0.0;
    const double off = 2.0 * kLseOff + 1e-15 * (__builtin_fabs(base) + __builtin_fabs(minus));
    int at = 0;
    uint64_t key = mine > 0 ? lists[lane * n] : 0ull, unsure = 0ull;
    double head = mine > 0 ? base + ((double)beam_logit(key) - minus) : kNone, last = kNone;
    int from = -1, written = 0;
    for (int i = 0; i <= n; ++i) {
      const double best = wave_reduce(head, kNone, [](double u, double v) { return u > v ? u : v; });
      if (!(best > kNone)) break;
      const int beam = __builtin_ctzll(__ballot(head == best));
      // every head of another beam than the last one's, so near to it that either may come first
      const uint64_t near = from < 0 ? 0ull : __ballot(lane != from && head > kNone && last - head <= off);
      if (near) unsure |= near | 1ull << from;
      if (i == n) break;
      if (lane == beam) {
        a.parent[at_out + i] = lane;
        a.token[at_out + i] = beam_id(key);
        a.score[at_out + i] = (float)head;
        a.out_finished[at_out + i] = ended || beam_id(key) == a.end_token ? 1 : 0;
        ++at;
        key = at < mine ? lists[lane * n + at] : 0ull;
        head = at < mine ? base + ((double)beam_logit(key) - minus) : kNone;
      }
      last = best;
      from = beam;
      written = i + 1;
    }
    for (int i = written + lane; i < n; i += 64) {
      a.parent[at_out + i] = -1;
      a.token[at_out + i] = 0;
      a.score[at_out + i] = -__builtin_inff();
      a.out_finished[at_out + i] = 0;
    }
    if (lane == 0) {
      a.len[q] = written;
      a.status[q] = status;
    }
    return unsure;
  };
  if (wave == 0) {
    uint64_t unsure = merge();
    unsure &= ~__ballot(ended);  // (a finished beam's score is exact)
    if (lane == 0) again = unsure;
  }
  __syncthreads();
  const uint64_t todo = again;
  if (todo) {  // (uniform)
    for (int b = 0; b < a.beams; ++b) {
      if (!(todo >> b & 1ull)) continue;
      const double exact = beam_exact_lse<DT, NWV>(a, q * a.beams + b, row_m[b], scratch);
      if (threadIdx.x == 0) lse[b] = exact;
    }
    __syncthreads();
    if (wave == 0) (void)merge();
  }
}

}  // namespace dspark
