// Beam search's selection over beams and vocabulary (dspark_beam_select).
//
// Rows are cut into slices, one workgroup each, which reads its slice once
// into registers: its maximum and sum of exponentials, and the logits that may
// be among the row's best -- those that reach the n_out-th largest of its
// threads' maxima, or of 64 groups' of four.  A second kernel joins a request:
// its waves join their beams' slices into log-sum-exps, and its threads select
// among all beams' candidates.  The first kernel is bound by vector instructions
// and reading alike (256 requests of 8 beams, 0.45 GB of bf16 rows of 129,280
// ids: 94 us, 4.7 TB/s, 90 % of the cycles issue; 107 us while each thread picked
// its candidates out of its registers; float32 rows 5.4 TB/s); the second is a
// chain of one workgroup's latencies (8 us for one request of 4 beams, 11 us for
// 256 of 8, 25 us for 8 of 32 with 64 selected).
//
// Order.  Within a beam the order of scores is the order of logits, whatever
// the log-sum-exp.  Between beams it hangs on their log-sum-exps, which
// binary32 exponentials give to kLseOff at most: an exponent t in base 2 is
// rounded by |t| 2^-24, and as much again by half from log2(e), the hardware
// exponential is off by 2^-23, and a term is in six sums of a thread and six of
// a wave before binary64 takes them; the weights' mean |t| is below 18 for 2^20
// logits, so that is 2^-24 (0.7 * 1.5 * 18 + 2 + 12) = 1.96e-6.  Where two
// neighbours in the merged order of different beams lie closer than twice
// kLseOff, their beams' log-sum-exps are computed again in binary64 and what
// decides is compared again, one after the other by the request's workgroup:
// 22 to 25 us for each alike beam of 129,280 ids (two of one request 20 -> 61 us, of
// 256 requests 109 -> 164; all beams alike, 8 of them 207 us, 32 800, 64 1,610;
// random requests come so close once in some thousands).
#pragma once
#include "../logits/slices.hpp"
#include "../logits/top.hpp"

namespace dspark {

constexpr int kBeams = 64;      // beams of a request: a lane each
constexpr int kBeamOut = 128;   // candidates selected
constexpr double kLseOff = 2e-6;
// candidates of a slice's list that there is room for
__host__ __device__ constexpr int beam_cap(int n_out) { return 2 * n_out + 64; }
constexpr int kBeamCap = beam_cap(kBeamOut);

struct BeamPart {
  float m;              // the slice's maximum
  float sum[kSliceNW];  // of each wave: the sum of exponentials relative to it
  int32_t flags;        // 1: a NaN, 2: a +inf
  int32_t count;        // candidates in the slice's list
  int32_t reserved;
};

struct BeamArgs {
  TopArgs x;  // rows, their width, temperature 1
  const float* scores;
  const int32_t* finished;
  int beams, n_out, end_token;
  int64_t requests;
  int32_t *parent, *token, *out_finished, *len, *status;
  float* score;
  int slices, length, cap;  // of a row, of nearly equal length; candidates of a slice's list
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

// The largest 16-bit key that at least n of 64 groups' maxima (a lane's v)
// reach, or where n is much for them, of the 256 values themselves: n values
// do, too.  0 where there are fewer than n.
__device__ __forceinline__ uint32_t reached_by(uint4 v, int n) {
  uint32_t T = 0;
  const uint32_t a = v.x > v.y ? v.x : v.y, b = v.z > v.w ? v.z : v.w, m = a > b ? a : b;
  if (2 * n <= __builtin_popcountll(__ballot(m != 0u))) {  // (uniform)
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t up = T | (1u << bit);
      if (__builtin_popcountll(__ballot(m >= up)) >= n) T = up;
    }
  } else {
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t up = T | (1u << bit);
      const int reach = __builtin_popcountll(__ballot(v.x >= up)) + __builtin_popcountll(__ballot(v.y >= up)) +
                        __builtin_popcountll(__ballot(v.z >= up)) + __builtin_popcountll(__ballot(v.w >= up));
      if (reach >= n) T = up;
    }
  }
  return T;
}

// the sum of the exponentials of N logits relative to m, quads first
template <int N>
__device__ __forceinline__ float beam_exp_sum(const TopArgs& a, float m, const float (&x)[N]) {
  float sum[N / 4];
  if (reference_fits(a, m)) {  // (uniform)
    const float K = m * a.c;
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(x[l], a.c, -K));
      sum[l / 4] = l % 4 ? sum[l / 4] + w : w;
    }
  } else {
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const float w = __builtin_amdgcn_exp2f((x[l] - m) * a.c);
      sum[l / 4] = l % 4 ? sum[l / 4] + w : w;
    }
  }
  return N == 8 ? sum[0] + sum[N / 4 - 1] : sum[0];
}

// (Seven waves a SIMD: with the three registers more that leave it six, the case
// above takes 106 us instead of 100.)
template <int DT, int U>
__global__ void __launch_bounds__(kSliceBS, 7) beam_slice_kernel(BeamArgs a) {
  constexpr int N = kVec<DT>;
  __shared__ __align__(16) uint32_t most[kSliceBS];
  __shared__ uint64_t near[kSliceNW][kBeamCap];  // a wave's candidates
  __shared__ float wave_m[kSliceNW];
  __shared__ uint32_t any_flags, held, counts[kSliceNW];
  typedef typename El<DT>::T XT;
  int64_t r;
  int s;
  if (!row_slice(a.x.n, a.slices, r, s)) return;
  BeamPart& p = a.part[r * a.slices + s];
  const int start = s * a.length, end = a.x.V - start < a.length ? a.x.V - start : a.length, tid = (int)threadIdx.x;
  if (!beam_live(a, r)) return;  // (uniform; the join does not read its record)
  const XT* row = static_cast<const XT*>(a.x.x) + r * a.x.stride;
  Raw<DT, N> raw[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int v = (i * kSliceBS + tid) * N;
    if (v < end) {
      raw[i] = raw_vec<DT, N, true>(row + start, v, end);
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) raw[i].w[w] = DT == DSPARK_F32 ? 0xff800000u : 0xff80ff80u;
    }
  }
  if (tid == 0) any_flags = 0u;
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
  const float own_m = wave_reduce(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); });
  if (lane_id() == 0) wave_m[wave_id()] = own_m;
  __syncthreads();
  float M = wave_m[0];
#pragma unroll
  for (int w = 1; w < kSliceNW; ++w) M = __builtin_fmaxf(M, wave_m[w]);
  // the threshold, by every wave for itself: -inf is no candidate
  float t = top_key_value<DSPARK_BF16>(reached_by(*reinterpret_cast<const uint4*>(most + 4 * lane_id()), a.n_out));
  t = t >= -3.4028235e38f ? t : -3.4028235e38f;
  uint32_t n = 0;  // the wave's candidates (uniform); their order does not matter
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const uint64_t reach = __ballot(x[i][l] >= t);
      if (reach) {  // (uniform)
        const uint32_t at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(reach >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)reach, 0u));
        if (x[i][l] >= t && at < (uint32_t)a.cap) near[wave_id()][at] = beam_key(x[i][l], start + (i * kSliceBS + tid) * N + l);
        n += (uint32_t)__builtin_popcountll(reach);
      }
    }
  }
  if (lane_id() == 0) counts[wave_id()] = n;
  const float ref = M == -__builtin_inff() ? 0.0f : M;
  float sum_of[U];
#pragma unroll
  for (int i = 0; i < U; ++i) sum_of[i] = beam_exp_sum(a.x, ref, x[i]);
#pragma unroll
  for (int d = 1; d < U; d *= 2) {
#pragma unroll
    for (int i = 0; i < U; i += 2 * d) sum_of[i] += sum_of[i + d];
  }
  float sum = sum_of[0];
  if (sum != sum || M == __builtin_inff()) {  // a NaN or a +inf in this thread, or the slice's
    uint32_t flags = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int l = 0; l < N; ++l) flags |= x[i][l] != x[i][l] ? 1u : x[i][l] == __builtin_inff() ? 2u : 0u;
    }
    if (flags) atomicOr(&any_flags, flags);
  }
  sum = wave_sum(sum);
  if (lane_id() == 63) p.sum[wave_id()] = sum;
  __syncthreads();
  uint64_t* list = a.cand + (r * a.slices + s) * a.cap;
  uint32_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kSliceNW; ++w) {
    if (w < wave_id()) before += counts[w];
    total += counts[w];
  }
  if (tid == 0) {
    p.m = M;
    p.flags = (int32_t)any_flags;
    p.count = total <= (uint32_t)a.cap ? (int)total : a.n_out;
  }
  if (total <= (uint32_t)a.cap) {  // (uniform)
    for (uint32_t i = (uint32_t)lane_id(); i < n; i += 64) list[before + i] = near[wave_id()][i];
    return;
  }
  // too many (equal logits): the largest logit that n_out reach, then of its
  // equals the lowest ids, each by halving (uniform; sums over the workgroup)
  const auto reaching = [&](auto reaches) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int l = 0; l < N; ++l) mine += (uint32_t)__builtin_popcountll(__ballot(reaches(x[i][l], (i * kSliceBS) * N + l)));
    }
    __syncthreads();
    if (lane_id() == 0) counts[wave_id()] = mine;
    __syncthreads();
    uint32_t sum_of = 0;
#pragma unroll
    for (int w = 0; w < kSliceNW; ++w) sum_of += counts[w];
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)sum_of);
  };
  // keys: one that n_out reach, and the largest that they may
  uint32_t low = (uint32_t)__builtin_amdgcn_readfirstlane((int)key32(t)), high = (uint32_t)__builtin_amdgcn_readfirstlane((int)key32(M));
  while (low < high) {
    const uint32_t mid = low + ((high - low) >> 1) + 1;
    const float f = top_key_value<DSPARK_F32>(mid);
    if (reaching([&](float v, int) { return v >= f; }) >= (uint32_t)a.n_out) low = mid;
    else high = mid - 1;
  }
  float f = top_key_value<DSPARK_F32>(low);
  const uint32_t equal = (uint32_t)a.n_out - reaching([&](float v, int) { return v > f; });
  int from = 0, to = a.length;  // ids below which fewer than `equal` of them lie, or as many
  while (to - from > 1) {
    const int mid = from + ((to - from) >> 1);
    asm volatile("" : "+v"(f));  // (comparisons with it are not to be kept over the rounds)
    if (reaching([&](float v, int id) { return v == f && tid * N < mid - id; }) >= equal) to = mid;
    else from = mid;
  }
  if (tid == 0) held = 0u;
  __syncthreads();
  asm volatile("" : "+v"(f));
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const int id = (i * kSliceBS + tid) * N + l;
      if (x[i][l] > f || (x[i][l] == f && id < to)) {
        const uint32_t place = atomicAdd(&held, 1u);
        if (place < (uint32_t)a.cap) list[place] = beam_key(x[i][l], start + id);
      }
    }
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

// e^y of y <= 0, off by |y| 2^-52 of its value at most (the series of e^f on |f| <= ln(2) / 2, up to f^12), 0 far below
__device__ __forceinline__ double beam_exp(double y) {
  const double t = (y > -1000.0 ? y : -1000.0) * 1.4426950408889634;
  const double n = __builtin_rint(t), f = (t - n) * 0.6931471805599453;
  double p = 1.0 / 479001600.0;
  constexpr double c[12] = {1.0,         1.0,          1.0 / 2.0,     1.0 / 6.0,      1.0 / 24.0,      1.0 / 120.0,
                            1.0 / 720.0, 1.0 / 5040.0, 1.0 / 40320.0, 1.0 / 362880.0, 1.0 / 3628800.0, 1.0 / 39916800.0};
#pragma unroll
  for (int i = 11; i >= 0; --i) p = __builtin_fma(p, f, c[i]);
  return __builtin_ldexp(p, (int)n);
}

// binary64 log-sum-exp of a row by the whole workgroup (every thread calls
// and gets it)
template <int DT, int NWV>
__device__ double beam_exact_lse(const BeamArgs& a, int64_t r, float M, double* scratch) {
  constexpr int N = kVec<DT>;
  const typename El<DT>::T* row = static_cast<const typename El<DT>::T*>(a.x.x) + r * a.x.stride;
  double sum = 0.0;
  constexpr int AT_ONCE = 8, STEP = NWV * 64 * N;  // vectors on their way
  for (int v0 = (int)threadIdx.x * N; v0 < a.x.V; v0 += AT_ONCE * STEP) {
    Raw<DT, N> raw[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j)
      if (v0 + j * STEP < a.x.V) raw[j] = raw_vec<DT, N, false>(row, v0 + j * STEP, a.x.V);
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (v0 + j * STEP >= a.x.V) break;
      float x[N];
      unpack<DT, N>(raw[j], x);
#pragma unroll
      for (int l = 0; l < N; ++l) sum += beam_exp((double)x[l] - (double)M);
    }
  }
  sum = group_reduce<NWV>(sum, 0.0, [](double u, double v) { return u + v; }, scratch);
  return (double)M + log(sum);
}

// The join's LDS: what a request's beams came to, and behind it either the
// candidates that may be among the best, or the beams' sorted lists.
constexpr int kBeamNear = 1024;  // candidates held
struct BeamScratch {
  double lse[kBeams];
  float m[kBeams], score[kBeams];
  int32_t n_list[kBeams], flags[kBeams];
  bool ended[kBeams];
  double red[16];
  uint16_t count[kBeams * kBeamSlices];  // of every slice's list
  uint32_t unsure[2], near, n_worth;
};
struct BeamNear {
  uint64_t key[kBeamNear];
  union {
    double score[kBeamNear];
    uint16_t worth[4 * kBeamNear];  // before the scores: the lists worth looking at
  };
  uint16_t order[kBeamNear];
  uint8_t beam[kBeamNear];
};  // behind it, the order key of every slice's best score (its upper half)
constexpr size_t beam_lists_bytes(int beams, int n_out, int waves) {
  return (size_t)beams * (size_t)n_out * 8 + (size_t)waves * (kBeamOut * 8 + (kBeamSlices + 2) * 4);
}
inline size_t beam_join_bytes(int beams, int slices, int n_out, int waves) {
  const size_t near = sizeof(BeamNear) + (size_t)beams * (size_t)slices * 2, lists = beam_lists_bytes(beams, n_out, waves);
  return near > lists ? near : lists;
}

__device__ __forceinline__ double beam_off(const BeamScratch& sh, int b) {
  return kLseOff + 1e-15 * (__builtin_fabs((double)sh.score[b]) + __builtin_fabs(sh.lse[b]));
}
__device__ __forceinline__ void beam_put(const BeamArgs& a, int64_t at, int beam, uint64_t key, double score, bool ended) {
  a.parent[at] = beam;
  a.token[at] = beam_id(key);
  a.score[at] = (float)score;
  a.out_finished[at] = ended || beam_id(key) == a.end_token ? 1 : 0;
}
__device__ __forceinline__ void beam_put_empty(const BeamArgs& a, int64_t at) {
  a.parent[at] = -1;
  a.token[at] = 0;
  a.score[at] = -__builtin_inff();
  a.out_finished[at] = 0;
}

// The log-sum-exps of the beams in `todo` again in binary64.
template <int DT, int NWV>
__device__ void beam_exact(const BeamArgs& a, int64_t q, uint64_t todo, BeamScratch& sh) {
  for (int b = 0; b < a.beams; ++b) {
    if (!(todo >> b & 1ull)) continue;
    const double exact = beam_exact_lse<DT, NWV>(a, q * a.beams + b, sh.m[b], sh.red);
    if (threadIdx.x == 0) sh.lse[b] = exact;
  }
  __syncthreads();
}

// The general way: each beam's best in a sorted list, by its wave, then one
// wave merges the lists, a beam to a lane.
template <int DT, int NWV>
__device__ void beam_join_lists(const BeamArgs& a, int64_t q, BeamScratch& sh, uint64_t* lists) {
  const int lane = lane_id(), wave = wave_id(), n = a.n_out;
  uint64_t* kept = lists + a.beams * n + wave * kBeamOut;
  uint32_t* first = reinterpret_cast<uint32_t*>(lists + a.beams * n + NWV * kBeamOut) + wave * (kBeamSlices + 2);
  for (int b = wave; b < a.beams; b += NWV) {  // (uniform in the wave)
    if (sh.ended[b]) {
      if (lane == 0) lists[b * n] = beam_key(0.0f, a.end_token);  // a score of its own: s + (0 - 0)
      continue;
    }
    const int64_t r = q * a.beams + b;
    const uint32_t c0 = 2 * lane < a.slices ? sh.count[b * a.slices + 2 * lane] : 0u;
    const uint32_t c1 = 2 * lane + 1 < a.slices ? sh.count[b * a.slices + 2 * lane + 1] : 0u;
    const uint32_t inc = wave_incl_scan(c0 + c1);
    first[2 * lane] = inc - c0 - c1;
    first[2 * lane + 1] = inc - c1;
    if (lane == 63) first[kBeamSlices] = inc;
    wave_sync();
    const int count = sh.n_list[b] ? (int)first[kBeamSlices] : 0;
    int held = 0;
    for (int g0 = 0; g0 < count; g0 += (kBeamPer - 2) * 64) {
      uint64_t key[kBeamPer];
#pragma unroll
      for (int j = 0; j < 2; ++j) key[j] = j * 64 + lane < held ? kept[j * 64 + lane] : 0ull;  // the best so far
#pragma unroll
      for (int j = 2; j < kBeamPer; ++j) {
        const int g = g0 + (j - 2) * 64 + lane;
        key[j] = 0ull;
        if (g < count) {
          int lo = 0, hi = a.slices - 1;  // the last slice that starts at or before g
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= (uint32_t)g) lo = mid;
            else hi = mid - 1;
          }
          key[j] = a.cand[(r * a.slices + lo) * a.cap + g - first[lo]];
        }
      }
      const uint64_t least = beam_cut(key, n, &held);
      int before = 0;
      wave_sync();
#pragma unroll
      for (int j = 0; j < kBeamPer; ++j) {
        const uint64_t in = __ballot(key[j] >= least);
        if (key[j] >= least) kept[before + __builtin_popcountll(in & ((1ull << lane) - 1ull))] = key[j];
        before += __builtin_popcountll(in);
      }
      wave_sync();
    }
    // sorted: an entry's place is the number of larger ones
#pragma unroll
    for (int j = 0; j < kBeamOut / 64; ++j) {
      const int e = j * 64 + lane;
      if (j * 64 < held) {  // (uniform)
        const uint64_t own = e < held ? kept[e] : 0ull;
        int larger = 0;
        for (int i = 0; i < held; ++i) larger += kept[i] > own ? 1 : 0;
        if (e < held) lists[b * n + larger] = own;
      }
    }
    if (lane == 0) sh.n_list[b] = held;
  }
  __syncthreads();

  const int64_t at_out = q * n;
  const auto merge = [&]() {  // by the first wave; the beams whose order is not certain
    constexpr double kNone = -__builtin_inf();
    const bool here = lane < a.beams;
    const int mine = here ? sh.n_list[lane] : 0;
    const double base = here ? (double)sh.score[lane] : 0.0, minus = here ? sh.lse[lane] : 0.0;
    const double off = here ? beam_off(sh, lane) : 0.0;
    int at = 0;
    uint64_t key = mine > 0 ? lists[lane * n] : 0ull, unsure = 0ull;
    double head = mine > 0 ? base + ((double)beam_logit(key) - minus) : kNone, last = kNone;
    int from = -1, written = 0;
    for (int i = 0; i <= n; ++i) {
      const double best = wave_reduce(head, kNone, [](double u, double v) { return u > v ? u : v; });
      if (!(best > kNone)) break;
      const int beam = __builtin_ctzll(__ballot(head == best));
      // every head of another beam than the last one's, so near to it that either may come first
      const uint64_t close = from < 0 ? 0ull : __ballot(lane != from && head > kNone && last - head <= off + beam_off(sh, from));
      if (close) unsure |= close | 1ull << from;
      if (i == n) break;
      if (lane == beam) {
        beam_put(a, at_out + i, lane, key, head, sh.ended[lane]);
        ++at;
        key = at < mine ? lists[lane * n + at] : 0ull;
        head = at < mine ? base + ((double)beam_logit(key) - minus) : kNone;
      }
      last = best;
      from = beam;
      written = i + 1;
    }
    for (int i = written + lane; i < n; i += 64) beam_put_empty(a, at_out + i);
    if (lane == 0) a.len[q] = written;
    return unsure & ~__ballot(here && sh.ended[lane]);  // (a finished beam's score is exact)
  };
  if (wave == 0) {
    const uint64_t unsure = merge();
    if (lane == 0) {
      sh.unsure[0] = (uint32_t)unsure;
      sh.unsure[1] = (uint32_t)(unsure >> 32);
    }
  }
  __syncthreads();
  const uint64_t todo = (uint64_t)sh.unsure[1] << 32 | sh.unsure[0];
  if (todo) {  // (uniform)
    beam_exact<DT, NWV>(a, q, todo, sh);
    if (wave == 0) (void)merge();
  }
}

// One workgroup per request.  Every slice's best logit is a candidate, so the
// n_out-th largest of their scores is a threshold (of few slices, the
// n_out-th largest of the threads' best candidates): the lists whose best reach
// it are few, and so are the candidates on them that do, which are sorted by
// counting.  Where they are not few (many equal scores), the beams' lists are
// merged instead.
template <int DT, int NWV>
__global__ void __launch_bounds__(64 * NWV) beam_join_kernel(BeamArgs a) {
  extern __shared__ __align__(16) uint64_t lists[];
  __shared__ BeamScratch sh;
  BeamNear& near = *reinterpret_cast<BeamNear*>(lists);
  uint16_t* best = reinterpret_cast<uint16_t*>(&near + 1);  // (0: none)
  const auto half = [](float x) -> uint16_t { return (uint16_t)(key32(x) >> 16); };
  const int64_t q = block_number(a.requests);
  if (q < 0) return;
  const int lane = lane_id(), wave = wave_id(), tid = (int)threadIdx.x, n = a.n_out;
  for (int b = wave; b < a.beams; b += NWV) {  // (uniform in the wave)
    const int64_t r = q * a.beams + b;
    // everything on its way at once (the records of a beam that takes no part hold nothing, and are not used)
    const BeamPart* part = a.part + r * a.slices;
    const float s = a.scores[r];
    const int32_t fin = a.finished ? a.finished[r] : 0;
    const BeamPart p0 = part[lane < a.slices ? lane : 0], p1 = part[64 + lane < a.slices ? 64 + lane : 0];
    if (!(__builtin_fabsf(s) < __builtin_inff()) || fin != 0) {
      const bool bad = s != s || s == __builtin_inff(), ended = fin != 0 && !bad && s > -__builtin_inff();
      if (lane == 0) {
        sh.flags[b] = bad ? 4 : 0;
        sh.n_list[b] = ended ? 1 : 0;
        sh.ended[b] = ended;
        sh.score[b] = s;
        sh.lse[b] = 0.0;
        sh.m[b] = 0.0f;
      }
      for (int i = lane; i < a.slices; i += 64) {
        sh.count[b * a.slices + i] = 0;
        best[b * a.slices + i] = ended && i == 0 ? half(s) : 0;
      }
      continue;
    }
    constexpr float kNone = -__builtin_inff();
    uint32_t f = 0u;
    float m[2] = {kNone, kNone};
    double sum[2] = {0.0, 0.0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // two slices to a lane
      const int i = j * 64 + lane;
      const BeamPart& p = j ? p1 : p0;
      if (i < a.slices) {
        sh.count[b * a.slices + i] = (uint16_t)p.count;
        f |= (uint32_t)p.flags;
        m[j] = p.m;
#pragma unroll
        for (int w = 0; w < kSliceNW; ++w) sum[j] += (double)p.sum[w];
      }
    }
    f = wave_reduce(f, 0u, [](uint32_t u, uint32_t v) { return u | v; });
    const float M = wave_reduce(__builtin_fmaxf(m[0], m[1]), kNone, [](float u, float v) { return __builtin_fmaxf(u, v); });
    double lse = 0.0;
    if (!f && M > kNone) {  // (uniform)
      const double top = sum_reference(a.x, M);
      double total = m[0] > kNone ? sum[0] * exp(sum_reference(a.x, m[0]) - top) : 0.0;
      if (a.slices > 64 && m[1] > kNone) total += sum[1] * exp(sum_reference(a.x, m[1]) - top);
      lse = top + log(wave_sum(total));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      // (a score below binary32 counts as its lowest value: the half key of -inf stands for no number)
      if (j * 64 + lane < a.slices)
        best[b * a.slices + j * 64 + lane] = m[j] > kNone ? half(__builtin_fmaxf((float)((double)s + ((double)m[j] - lse)), -3.4028235e38f)) : 0;
    if (lane == 0) {
      sh.flags[b] = (int)f;
      sh.n_list[b] = M > kNone ? 1 : 0;
      sh.ended[b] = false;
      sh.score[b] = s;
      sh.lse[b] = lse;
      sh.m[b] = M;
    }
  }
  if (tid == 0) {
    sh.unsure[0] = sh.unsure[1] = 0u;
    sh.near = sh.n_worth = 0u;
  }
  __syncthreads();
  const uint32_t bad = wave_reduce(lane < a.beams ? (uint32_t)sh.flags[lane] : 0u, 0u, [](uint32_t u, uint32_t v) { return u | v; });
  const int64_t at_out = q * n;
  if (tid == 0)
    a.status[q] = bad & 1u ? DSPARK_ST_ROW_NAN : bad & 2u ? DSPARK_ST_ROW_POSINF : bad & 4u ? DSPARK_ST_BAD_SCORE : DSPARK_ST_OK;
  if (bad) {  // (uniform)
    for (int i = tid; i < n; i += 64 * NWV) beam_put_empty(a, at_out + i);
    if (tid == 0) a.len[q] = 0;
    return;
  }

  // candidates of `total` lists, the w-th of them list_of(w): 16, 32 or 64
  // threads to a list, two keys to a thread, two lists at a time
  const int n_lists = a.beams * a.slices, shift = n <= 12 ? 4 : n <= 28 ? 5 : 6, width = 1 << shift, groups = 64 * NWV >> shift;
  const int e0 = tid & (width - 1);
  const auto score_of = [&](int b, uint64_t key) { return (double)sh.score[b] + ((double)beam_logit(key) - sh.lse[b]); };
  const auto each = [&](int total, auto list_of, auto take) {
    for (int w0 = tid >> shift; w0 < total; w0 += 2 * groups) {
      uint64_t key[2][2];
      int L[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        L[i] = w0 + i * groups < total ? list_of(w0 + i * groups) : -1;
        const int c = L[i] >= 0 ? sh.count[L[i]] : 0;
        const uint64_t* list = a.cand + (q * n_lists + L[i]) * a.cap;
#pragma unroll
        for (int j = 0; j < 2; ++j) key[i][j] = e0 + j * width < c ? list[e0 + j * width] : 0ull;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!key[i][0]) continue;
        const int b = (int)((uint32_t)L[i] / (uint32_t)a.slices), c = sh.count[L[i]];
        take(b, key[i][0]);
        if (key[i][1]) take(b, key[i][1]);
        for (int e = e0 + 2 * width; e < c; e += width) take(b, a.cand[(q * n_lists + L[i]) * a.cap + e]);
      }
    }
    if (tid < a.beams && sh.ended[tid]) take(tid, beam_key(0.0f, a.end_token));
  };

  // the threshold: the largest half key that n of the lists' best reach (512
  // of them, or groups of lists); where there are few lists, that n threads'
  // best do
  static_assert(NWV == 8, "eight groups of lists to a lane");
  uint32_t T = 0;
  {
    uint32_t v[NWV];
    if (n_lists >= 4 * n) {  // (uniform)
#pragma unroll
      for (int i = 0; i < NWV; ++i) {
        v[i] = 0u;
        for (int L = i * 64 + lane; L < n_lists; L += 64 * NWV) v[i] = best[L] > v[i] ? best[L] : v[i];
      }
    } else {
      float top = -__builtin_inff();
      each(n_lists, [](int w) { return w; }, [&](int b, uint64_t key) { top = __builtin_fmaxf(top, (float)score_of(b, key)); });
      near.order[tid] = top > -__builtin_inff() ? half(top) : 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NWV; ++i) v[i] = near.order[i * 64 + lane];
    }
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t up = T | (1u << bit);
      int reach = 0;
#pragma unroll
      for (int i = 0; i < NWV; ++i) reach += __builtin_popcountll(__ballot(v[i] >= up));
      if (reach >= n) T = up;
    }
  }
  // n candidates' scores reach it as they were computed: those of the best do
  // so but for what the log-sum-exps are off, and a rounding
  float t = top_key_value<DSPARK_BF16>(T);
  t = T ? t - (1e-5f + __builtin_fabsf(t) * 0x1p-20f) : -__builtin_inff();
  const uint32_t least = T ? half(t) : 1u;
  for (int L = tid; L < n_lists; L += 64 * NWV) {
    if (best[L] >= least && sh.count[L] != 0) {
      const uint32_t at = atomicAdd(&sh.n_worth, 1u);
      if (at < 4u * kBeamNear) near.worth[at] = (uint16_t)L;
    }
  }
  __syncthreads();
  const int n_worth = (int)sh.n_worth;
  const auto take = [&](int b, uint64_t key) {
    if (!((float)score_of(b, key) >= t)) return;
    const uint32_t at = atomicAdd(&sh.near, 1u);
    if (at < (uint32_t)kBeamNear) {
      near.key[at] = key;
      near.beam[at] = (uint8_t)b;
    }
  };
  if (n_worth <= 4 * kBeamNear) each(n_worth, [&](int w) { return (int)near.worth[w]; }, take);
  __syncthreads();
  const int count = (int)sh.near;
  if (count > kBeamNear || n_worth > 4 * kBeamNear) {  // (uniform)
    __syncthreads();
    beam_join_lists<DT, NWV>(a, q, sh, lists);
    return;
  }
  const int out = count < n ? count : n;
  const auto sort = [&]() {  // a place is the number of better ones: score, then beam, then logit and id
    for (int i = tid; i < count; i += 64 * NWV) near.score[i] = score_of(near.beam[i], near.key[i]);
    __syncthreads();
    for (int i = tid >> 2; i < count; i += 16 * NWV) {  // four threads to a candidate
      const double own = near.score[i];
      const int beam = near.beam[i];
      const uint64_t key = near.key[i];
      uint32_t better = 0;
      for (int j = tid & 3; j < count; j += 4) {
        const double o = near.score[j];
        const int ob = near.beam[j];
        better += o > own || (o == own && (ob < beam || (ob == beam && near.key[j] > key))) ? 1u : 0u;
      }
      better += dpp_u32<0xb1, 0xf, 0xf>(better, better);  // quad_perm 1,0,3,2
      better += dpp_u32<0x4e, 0xf, 0xf>(better, better);  // quad_perm 2,3,0,1
      if ((tid & 3) == 0) near.order[better] = (uint16_t)i;
    }
    __syncthreads();
  };
  sort();
  // neighbours of two beams, so near to each other that either may come first
  for (int i = tid; i + 1 < count; i += 64 * NWV) {
    const int x = near.order[i], y = near.order[i + 1], bx = near.beam[x], by = near.beam[y];
    const double off = beam_off(sh, bx) + beam_off(sh, by);
    if (bx != by && near.score[x] - near.score[y] <= off && (i < n || near.score[near.order[n - 1]] - near.score[x] <= off)) {
      if (!sh.ended[bx]) atomicOr(&sh.unsure[bx >> 5], 1u << (bx & 31));
      if (!sh.ended[by]) atomicOr(&sh.unsure[by >> 5], 1u << (by & 31));
    }
  }
  __syncthreads();
  const uint64_t todo = (uint64_t)sh.unsure[1] << 32 | sh.unsure[0];
  if (todo) {  // (uniform)
    beam_exact<DT, NWV>(a, q, todo, sh);
    sort();
  }
  for (int i = tid; i < n; i += 64 * NWV) {
    if (i < out) {
      const int x = near.order[i];
      beam_put(a, at_out + i, near.beam[x], near.key[x], near.score[x], sh.ended[near.beam[x]]);
    } else {
      beam_put_empty(a, at_out + i);
    }
  }
  if (tid == 0) a.len[q] = out;
}

}  // namespace dspark
