// The top logits of a row with the log-sum-exp of the whole row
// (dspark_top_logits).
//
// Long rows (and many rows of middle length) are cut into slices of 8,192
// ids, one workgroup each, which reads its slice once into registers.  A threshold that the k-th
// largest logit lies above with good odds comes from a sample of the row
// (2,048 logits, the same for every slice of the row), so that one pass
// yields the slice's maximum, its sum of exponentials and the few logits
// that may be among the top k.  A second kernel joins the slices of a row and
// selects exactly among those candidates.  A row whose candidates are too
// few or too many for their list (heavy ties, a sample that misleads) is
// selected from memory by that kernel's workgroup instead: slower, the same
// answer.  Other rows are held whole in one workgroup's registers.  1,280 bf16
// rows of V = 129,280 take 71 + 12 us (4.7 TB/s of their bytes while they are
// read), 320 float32 rows 36 + 11.
//
// Exponentials are exp2(x c - K), one fused multiply-add each, with c the
// binary32 rounding of log2(e) / T and K = c times a maximum: the reference
// K is exact as it stands (the sum is over 2^(x c) / 2^K), and what the
// rounding of c does to the row's largest logits is put back in binary64
// (sum_reference).  The exponent of the maximum itself is then K's own rounding,
// half its last place: 2 at |K| = 2^26, but hundreds from 2^32 on (logits of 1e9
// and more, or temperatures below 2^-26), where the exponential overflows or
// vanishes.  From 2^26 on they are exp2((x - m) c), exactly 1 at the maximum.
#pragma once
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
  float c;  // binary32 log2(e) / T
  int32_t* ids;
  float* logits;
  int32_t* len;
  float* lse;
  int32_t* row_status;
};

constexpr double kLn2 = 0.69314718055994530942;

// k of row r: -1 when out of range
__device__ __forceinline__ int row_k(const TopArgs& a, int64_t r) {
  const int cap = a.k_max < a.V ? a.k_max : a.V;
  const int k = a.topk ? a.topk[r] : cap;
  return k < 0 || k > cap ? -1 : k;
}

// whether the rounding of K = m c stays within 2 (see above)
__device__ __forceinline__ bool reference_fits(const TopArgs& a, float m) { return __builtin_fabsf(m) * a.c < 0x1p26f; }
// log of what a sum of exponentials relative to the maximum m is to be multiplied by
__device__ __forceinline__ double sum_reference(const TopArgs& a, float m) {
  if (!reference_fits(a, m)) return (double)m * a.inv_t;
  return (double)(m * a.c) * kLn2 + (a.inv_t - (double)a.c * kLn2) * (double)m;
}
// the sum of the exponentials of N logits relative to the maximum m
template <int N>
__device__ __forceinline__ float exp_sum(const TopArgs& a, float m, const float (&x)[N]) {
  float sum = 0.0f;
  if (reference_fits(a, m)) {  // (uniform)
    const float K = m * a.c;
#pragma unroll
    for (int l = 0; l < N; ++l) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(x[l], a.c, -K));
  } else {
#pragma unroll
    for (int l = 0; l < N; ++l) sum += __builtin_amdgcn_exp2f((x[l] - m) * a.c);
  }
  return sum;
}

__device__ __forceinline__ int top_status(uint32_t flags, float m, int k) {
  return flags & 1u ? DSPARK_ST_ROW_NAN
         : flags & 2u ? DSPARK_ST_ROW_POSINF
         : m == -__builtin_inff() ? DSPARK_ST_ROW_ZERO_MASS
         : k < 0 ? DSPARK_ST_BAD_TOPK : DSPARK_ST_OK;
}

template <int DT>
__device__ __forceinline__ uint32_t top_key(float x) {  // order-preserving, 0 below every finite logit's
  return DT == DSPARK_BF16 ? key32(x) >> 16 : key32(x);
}
template <int DT>
__device__ __forceinline__ float top_key_value(uint32_t k) {  // the smallest value with that key
  const uint32_t b = DT == DSPARK_BF16 ? k << 16 : k;
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}

constexpr int kTopBins = 2048;

// Scratch of a selection by NWV waves.
template <int NWV>
struct TopScratch {
  uint32_t hist[kTopBins];
  uint32_t scan[NWV];
  double red[NWV];
  uint32_t bin, above;
  uint32_t few[64], n_few;  // the keys of a bin that holds few
};

// The bin where the running count from bin 0 on reaches `need` (which the
// bins hold at least), and the count of the bins before it.
template <int NWV>
__device__ __forceinline__ uint32_t top_crossing(TopScratch<NWV>& sh, uint32_t need, uint32_t* above) {
  constexpr int PER = kTopBins / (64 * NWV);
  uint32_t c[PER], sum = 0, total;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = sh.hist[threadIdx.x * PER + i];
    sum += c[i];
  }
  uint32_t run = group_excl_scan<NWV>(sum, sh.scan, &total);
  if (run < need && need <= run + sum) {
    int hit = -1;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (hit < 0) {
        if (run + c[i] >= need) {
          hit = i;
          sh.bin = threadIdx.x * PER + i;
          sh.above = run;
        }
        run += c[i];
      }
    }
  }
  __syncthreads();
  *above = sh.above;
  return sh.bin;
}

// The n largest keys (1 <= n <= how many there are; key 0: none): every key
// above T and, of the keys equal to T, the first `ties` by id.
struct TopCut {
  uint32_t T, ties;
};

// Cut among keys held PER to a thread, all of them 0 or in [lo, hi]:
// histograms of a range, narrowed to one key or to a bin taken whole.
template <int NWV, int PER>
__device__ __forceinline__ TopCut top_cut(const uint32_t (&key)[PER], uint32_t lo, uint32_t hi, uint32_t n, TopScratch<NWV>& sh) {
  for (;;) {
    const uint32_t range = hi - lo;
    const int shift = range < (uint32_t)kTopBins ? 0 : (32 - __builtin_clz(range)) - 11;
    for (int i = threadIdx.x; i < kTopBins; i += 64 * NWV) sh.hist[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] >= lo && key[j] <= hi) atomicAdd(&sh.hist[(hi - key[j]) >> shift], 1u);
    __syncthreads();
    uint32_t above;
    const uint32_t bin = top_crossing<NWV>(sh, n, &above);
    n -= above;
    const uint32_t held = sh.hist[bin];
    const uint32_t bhi = hi - (bin << shift), width = (1u << shift) - 1u;
    const uint32_t blo = bhi - lo > width ? bhi - width : lo;
    __syncthreads();
    if (held == n) return TopCut{blo - 1u, 0u};  // all keys from blo on (blo >= 1)
    if (shift == 0) return TopCut{bhi, n};
    if (held <= 64u) {  // one wave ranks them
      if (threadIdx.x == 0) sh.n_few = 0u;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (key[j] >= blo && key[j] <= bhi) sh.few[atomicAdd(&sh.n_few, 1u)] = key[j];
      __syncthreads();
      if (wave_id() == 0) {
        const uint32_t own = (uint32_t)lane_id() < held ? sh.few[lane_id()] : 0u;
        uint32_t more = 0, same = 0;
        for (uint32_t i = 0; i < held; ++i) {
          const uint32_t o = sh.few[i];
          more += o > own ? 1u : 0u;
          same += o == own ? 1u : 0u;
        }
        if (own && more < n && n <= more + same) {  // (every lane that holds the key: the same values)
          sh.bin = own;
          sh.above = n - more;
        }
      }
      __syncthreads();
      return TopCut{sh.bin, sh.above};
    }
    hi = bhi;
    lo = blo;
  }
}

// Writes the chosen ones of a thread-major list in its order, zeros behind
// them up to k_max.
template <int NWV, int PER, class ID, class VALUE>
__device__ __forceinline__ void top_write(const TopArgs& a, int64_t r, const uint32_t (&key)[PER], TopCut cut, int n,
                                          TopScratch<NWV>& sh, ID id, VALUE value) {
  uint32_t cnt = 0, total;  // low half: above the cut, high half: ties (each at most PER 64 NWV <= 2^14)
#pragma unroll
  for (int j = 0; j < PER; ++j) cnt += key[j] > cut.T ? 1u : key[j] == cut.T && cut.T ? 0x10000u : 0u;
  uint32_t pre = group_excl_scan<NWV>(cnt, sh.scan, &total);
  int32_t* ids = a.ids + r * a.k_max;
  float* logits = a.logits + r * a.k_max;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool sure = key[j] > cut.T, tie = !sure && key[j] == cut.T && cut.T;
    const uint32_t tb = pre >> 16;
    if (sure || (tie && tb < cut.ties)) {
      const uint32_t pos = (pre & 0xffffu) + (tb < cut.ties ? tb : cut.ties);
      if (pos < (uint32_t)a.k_max) {
        ids[pos] = id(j);
        logits[pos] = value(j);
      }
    }
    pre += sure ? 1u : tie ? 0x10000u : 0u;
  }
  for (int e = n + (int)threadIdx.x; e < a.k_max; e += 64 * NWV) {
    ids[e] = 0;
    logits[e] = 0.0f;
  }
}

__device__ __forceinline__ void top_row_out(const TopArgs& a, int64_t r, int status, int n, float lse) {
  if (threadIdx.x != 0) return;
  const bool ok = status == DSPARK_ST_OK;
  a.row_status[r] = status;
  a.len[r] = ok ? n : 0;
  if (a.lse) a.lse[r] = ok ? lse : 0.0f;
}

// --------------------------------------------- rows selected from memory
// The top k of a good row whose candidates do not fit, by one workgroup:
// digit histograms over passes of the row, then an ordered pass that writes.
template <int DT, int NWV>
__device__ __forceinline__ int top_from_memory(const TopArgs& a, int64_t r, int k, TopScratch<NWV>& sh) {
  typedef typename El<DT>::T XT;
  const XT* row = static_cast<const XT*>(a.x) + r * a.stride;
  const int V = a.V;
  constexpr int N = kVec<DT>, kStep = 64 * NWV * N;
  const uint32_t none = top_key<DT>(-__builtin_inff());  // -inf is not listed
  uint32_t prefix = 0, pmask = 0, need = (uint32_t)k, n = (uint32_t)k;
  bool first = true;
  for (int shift = DT == DSPARK_BF16 ? 8 : 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < kTopBins; i += 64 * NWV) sh.hist[i] = 0u;
    __syncthreads();
    for (int v = (int)threadIdx.x * N; v < V; v += kStep) {
      float x[N];
      load_vec<DT, N>(row, v, V, x);
#pragma unroll
      for (int l = 0; l < N; ++l) {
        const uint32_t key = top_key<DT>(x[l]);
        const bool in = v + l < V && key > none && (key & pmask) == prefix;
        const uint32_t bin = 255u - ((key >> shift) & 255u);  // the largest digits first
        // equal logits meet in one bin: lanes that share the first lane's are counted together
        const uint64_t act = __ballot(in);
        if (!act) continue;
        const int lead = __builtin_ctzll(act);
        const uint32_t b0 = (uint32_t)__builtin_amdgcn_readlane((int)bin, lead);
        const uint64_t same = __ballot(in && bin == b0);
        if (lane_id() == lead) atomicAdd(&sh.hist[b0], (uint32_t)__builtin_popcountll(same));
        if (in && bin != b0) atomicAdd(&sh.hist[bin], 1u);
      }
    }
    __syncthreads();
    if (first) {  // fewer finite logits than k
      uint32_t mine = 0, total;
      for (int i = threadIdx.x; i < 256; i += 64 * NWV) mine += sh.hist[i];
      (void)group_excl_scan<NWV>(mine, sh.scan, &total);
      if (total < need) need = n = total;
      first = false;
    }
    uint32_t above;
    const uint32_t bin = top_crossing<NWV>(sh, need, &above);
    need -= above;
    prefix |= (255u - bin) << shift;
    pmask |= 255u << shift;
    __syncthreads();
  }
  // keys above the prefix and the first `need` equal to it, in id order
  uint32_t placed = 0, tied = 0;
  for (int base = 0; base < V; base += kStep) {
    const int v = base + (int)threadIdx.x * N;
    float x[N];
    if (v < V) load_vec<DT, N>(row, v, V, x);
    uint32_t cnt = 0, total;
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const uint32_t key = v + l < V ? top_key<DT>(x[l]) : 0u;
      cnt += key > prefix ? 1u : key == prefix ? 0x10000u : 0u;
    }
    uint32_t pre = group_excl_scan<NWV>(cnt, sh.scan, &total);
#pragma unroll
    for (int l = 0; l < N; ++l) {
      const uint32_t key = v + l < V ? top_key<DT>(x[l]) : 0u;
      const uint32_t tb = tied + (pre >> 16);
      if (key > prefix || (key == prefix && tb < need)) {
        const uint32_t pos = placed + (pre & 0xffffu) + (tb < need ? tb : need);
        if (pos < (uint32_t)a.k_max) {
          a.ids[r * a.k_max + pos] = v + l;
          a.logits[r * a.k_max + pos] = x[l];
        }
      }
      pre += key > prefix ? 1u : key == prefix ? 0x10000u : 0u;
    }
    placed += total & 0xffffu;
    tied += total >> 16;
  }
  for (int e = (int)n + (int)threadIdx.x; e < a.k_max; e += 64 * NWV) {
    a.ids[r * a.k_max + e] = 0;
    a.logits[r * a.k_max + e] = 0.0f;
  }
  return (int)n;
}

// ------------------------------------------------------------ short rows
constexpr int kTopSmall = 16384;  // 1,024 threads of 16 logits

// A row of at most 64 NWV 8 G ids in the workgroup's registers, 8 G
// neighbouring ones to a thread.
template <int DT, int NWV, int G>
__global__ void __launch_bounds__(64 * NWV) top_small_kernel(TopArgs a) {
  __shared__ TopScratch<NWV> sh;
  typedef typename El<DT>::T XT;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  const XT* row = static_cast<const XT*>(a.x) + r * a.stride;
  const int v0 = (int)threadIdx.x * 8 * G;
  float x[8 * G];
  float m = -__builtin_inff();
  uint32_t flags = 0;
  constexpr int N = kVec<DT>;
#pragma unroll
  for (int g = 0; g < 8 * G / N; ++g) {
    float y[N];
    load_vec<DT, N>(row, v0 + N * g, a.V, y);
#pragma unroll
    for (int l = 0; l < N; ++l) {
      x[N * g + l] = y[l];
      m = __builtin_fmaxf(m, y[l]);
      flags |= y[l] != y[l] ? 1u : y[l] == __builtin_inff() ? 2u : 0u;
    }
  }
  const float M = group_reduce<NWV>(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); },
                                    reinterpret_cast<float*>(sh.red));
  flags = group_reduce<NWV>(flags, 0u, [](uint32_t u, uint32_t v) { return u | v; }, sh.scan);
  const int k = row_k(a, r);
  const int status = top_status(flags, M, k);
  int n = 0;
  float lse = 0.0f;
  uint32_t key[8 * G];
  TopCut cut{0xffffffffu, 0u};
  if (status == DSPARK_ST_OK) {
    const float part = exp_sum(a, M, x);
    uint32_t fin = 0, total;
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) {
      key[j] = x[j] > -__builtin_inff() ? top_key<DT>(x[j]) : 0u;
      fin += key[j] ? 1u : 0u;
    }
    const double sum = group_reduce<NWV>((double)part, 0.0, [](double u, double v) { return u + v; }, sh.red);
    lse = (float)(sum_reference(a, M) + log(sum));
    (void)group_excl_scan<NWV>(fin, sh.scan, &total);
    n = (uint32_t)k < total ? k : (int)total;
    if (n > 0) cut = top_cut<NWV>(key, 1u, top_key<DT>(M), (uint32_t)n, sh);
  } else {
#pragma unroll
    for (int j = 0; j < 8 * G; ++j) key[j] = 0u;
  }
  top_write<NWV>(a, r, key, cut, n, sh, [&](int j) { return v0 + j; }, [&](int j) { return x[j]; });
  top_row_out(a, r, status, n, lse);
}

// ------------------------------------------------------- rows in slices
constexpr int kTopSlice = 4 * kSliceStep;                  // ids of a slice
constexpr int kTopSlices = DSPARK_V_MAX / kTopSlice;       // slices of the longest row
constexpr int kTopSample = kSliceBS * 8;                   // logits sampled of a row: 64 runs of 32

struct TopPart {
  float m[kSliceNW], sum[kSliceNW];  // of each wave: its maximum, the sum of exponentials relative to it
  float t;       // the row's threshold
  int32_t flags; // 1: a NaN, 2: a +inf
  int32_t count; // candidates (more than the list holds: too many)
  int32_t reserved;
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
};
template <>
struct Cand<DSPARK_F32> {
  typedef uint2 T;
  static __device__ __forceinline__ T make(float x, int t) { return make_uint2(__float_as_uint(x), (uint32_t)t); }
  static __device__ __forceinline__ float value(T c) { return __uint_as_float(c.x); }
  static __device__ __forceinline__ int place(T c) { return (int)c.y; }
};

struct TopSliceArgs {
  TopArgs a;
  int slices;
  int cap;      // candidates a slice's list holds
  int rank;     // the threshold is about the rank-th largest of the sample's 256 maxima
  TopPart* part;  // [n][slices]
  void* cand;     // [n][slices][cap]
};

// mask = 2 mask + (x >= t): a compare and an add with its carry
__device__ __forceinline__ void push_ge(uint32_t& mask, float x, float t) {
  asm("v_cmp_ge_f32 vcc, %1, %2\n\tv_addc_co_u32 %0, vcc, %0, %0, vcc" : "+v"(mask) : "v"(x), "v"(t) : "vcc");
}

// What bounds it is reading, though it is a quarter above what a copy's rate
// would give: without the exponentials (five of eleven cycles' issue per bf16
// logit) 1,280 bf16 rows take 65 us instead of 71, and an eighth fewer vector
// instructions around them changed nothing.  Each wave has a reference of its
// own, the order of the candidates comes from one scan of packed counts.  A
// candidate's logit is picked from a copy of the slice in LDS (read again from
// memory it held its wave up: 91 us instead of 71).
template <int DT>
__global__ void __launch_bounds__(kSliceBS) top_slice_kernel(TopSliceArgs q) {
  __shared__ __align__(16) uint32_t sample[kSliceBS];
  __shared__ float thr;
  constexpr int N = kVec<DT>, U = kTopSlice / (kSliceBS * N);  // U vectors per thread: 32 logits
  constexpr int W = U / 4;                                     // words of four 16-bit counts
  __shared__ uint64_t scan[W][kSliceNW];
  __shared__ uint32_t any_flags;
  typedef typename El<DT>::T XT;
  int64_t r;
  int s;
  if (!row_slice(q.a.n, q.slices, r, s)) return;
  const int start = s * kTopSlice, V = q.a.V, tid = (int)threadIdx.x;
  const XT* row = static_cast<const XT*>(q.a.x) + r * q.a.stride;
  const int run = (V / 64) & ~7;  // the sample: 64 runs of 32 logits, four threads each
  float smp[8], x[U][N];
  __shared__ __align__(16) uint32_t held[kTopSlice * sizeof(XT) / 4];  // the slice as it was loaded
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) {
    float y[N];
    load_whole<DT, N>(row, (tid >> 2) * run + (i * 4 + (tid & 3)) * N, y);
#pragma unroll
    for (int l = 0; l < N; ++l) smp[i * N + l] = y[l];
  }
  Raw<DT, N> raw[U];
  if (start + kTopSlice <= V) {  // (uniform)
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = raw_whole<DT, N, true>(row + start, (uint32_t)(i * kSliceBS + tid) * N);
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) raw[i] = raw_vec<DT, N, true>(row + start, (i * kSliceBS + tid) * N, V - start);
  }
  float top = smp[0];
#pragma unroll
  for (int l = 1; l < 8; ++l) top = __builtin_fmaxf(top, smp[l]);
  sample[tid] = top != top ? 0u : key32(top) >> 16;
  if (tid == 0) any_flags = 0u;
  __syncthreads();
  if (wave_id() == 0) {
    // the largest 16-bit key that at least `rank` of the maxima reach: four
    // maxima a lane, sixteen steps of ballots
    const uint4 o = *reinterpret_cast<const uint4*>(sample + 4 * lane_id());
    uint32_t T = 0;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t up = T | (1u << bit);
      const int reach = __builtin_popcountll(__ballot(o.x >= up)) + __builtin_popcountll(__ballot(o.y >= up)) +
                        __builtin_popcountll(__ballot(o.z >= up)) + __builtin_popcountll(__ballot(o.w >= up));
      if (reach >= q.rank) T = up;
    }
    // -inf is no candidate: the threshold is the lowest finite value at least
    const float t = top_key_value<DSPARK_BF16>(T);
    if (lane_id() == 0) thr = t >= -3.4028235e38f ? t : -3.4028235e38f;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    unpack<DT, N>(raw[i], x[i]);
    const uint4 w = make_uint4(raw[i].w[0], raw[i].w[1], raw[i].w[2], raw[i].w[3]);
    *reinterpret_cast<uint4*>(held + (i * kSliceBS + tid) * 4) = w;
  }
  float m = x[0][0];
#pragma unroll
  for (int i = 0; i < U; ++i) {
#pragma unroll
    for (int l = 0; l < N; ++l) m = __builtin_fmaxf(m, x[i][l]);
  }
  const float M = wave_reduce(m, -__builtin_inff(), [](float u, float v) { return __builtin_fmaxf(u, v); });
  const float ref = M == -__builtin_inff() ? 0.0f : M;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < U; ++i) sum += exp_sum(q.a, ref, x[i]);
  if (sum != sum || M == __builtin_inff()) {  // a NaN or a +inf in this thread, or the wave's
    uint32_t flags = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int l = 0; l < N; ++l) flags |= x[i][l] != x[i][l] ? 1u : x[i][l] == __builtin_inff() ? 2u : 0u;
    }
    if (flags) atomicOr(&any_flags, flags);
  }
  const float wsum = wave_sum(sum);
  __syncthreads();
  const float t = thr;
  uint32_t mask = 0;  // element l of vector i at bit N i + N - 1 - l
#pragma unroll
  for (int i = U - 1; i >= 0; --i) {
#pragma unroll
    for (int l = 0; l < N; ++l) push_ge(mask, x[i][l], t);
  }
  // places in the list: by vector, then thread, then element -- id order
  constexpr uint32_t kOnes = (1u << N) - 1u;
  TopPart& p = q.part[r * q.slices + s];
  uint64_t before[W];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint64_t count = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) count |= (uint64_t)__builtin_popcount((mask >> (N * (4 * w + i))) & kOnes) << (16 * i);
    const uint64_t inc = wave_incl_scan(count);
    before[w] = inc - count;
    if (lane_id() == 63) scan[w][wave_id()] = inc;
  }
  if (lane_id() == 63) {
    p.m[wave_id()] = M;
    p.sum[wave_id()] = wsum;
  }
  __syncthreads();
  typename Cand<DT>::T* list = static_cast<typename Cand<DT>::T*>(q.cand) + (r * q.slices + s) * q.cap;
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint64_t all = 0;
#pragma unroll
    for (int v = 0; v < kSliceNW; ++v) {
      const uint64_t o = scan[w][v];
      before[w] += v < wave_id() ? o : 0ull;
      all += o;
    }
    // the vectors before: every field stays below 2^14
    before[w] += (all << 16) + (all << 32) + (all << 48) + (uint64_t)base * 0x0001000100010001ull;
    base += (uint32_t)((all >> 48) + (all >> 32) + (all >> 16) + all) & 0xffffu;
    uint32_t left = W == 1 ? mask : (mask >> (16 * w)) & 0xffffu;
    while (left) {
      const int i = __builtin_ctz(left) / N;  // the lowest vector left
      const uint32_t own = (left >> (N * i)) & kOnes;
      const int l = __builtin_clz(own) - (32 - N);
      const uint32_t pos = (uint32_t)(before[w] >> (16 * i)) & 0xffffu;
      before[w] += 1ull << (16 * i);
      left &= ~((1u << (N - 1)) >> l << (N * i));
      const int place = ((4 * w + i) * kSliceBS + tid) * N + l;
      if (pos < (uint32_t)q.cap) list[pos] = Cand<DT>::make(El<DT>::get(reinterpret_cast<const XT*>(held), place), place);
    }
  }
  if (tid == 0) {
    p.t = t;
    p.flags = (int32_t)any_flags;
    p.count = (int32_t)base;
    p.reserved = 0;
  }
}

// One workgroup per row: joins its slices and selects among the candidates
// (at most kTopPer per thread).
template <int DT, int NWV, int kTopPer>
__global__ void __launch_bounds__(64 * NWV) top_select_kernel(TopSliceArgs q) {
  __shared__ TopScratch<NWV> sh;
  __shared__ uint32_t first[kTopSlices + 1];  // candidates before each slice
  __shared__ double row_sum;
  __shared__ float row_m;
  __shared__ uint32_t row_flags, row_over;
  const TopArgs& a = q.a;
  const int64_t r = block_number(a.n);
  if (r < 0) return;
  const TopPart* part = q.part + r * q.slices;
  if (wave_id() == 1) {  // the sums: one wave's record per lane
    const int l = lane_id();
    constexpr float kNone = -__builtin_inff();
    float m = kNone;
    for (int i = l; i < q.slices * kSliceNW; i += 64) m = __builtin_fmaxf(m, part[i / kSliceNW].m[i % kSliceNW]);
    const float M = wave_reduce(m, kNone, [](float u, float v) { return __builtin_fmaxf(u, v); });
    const double top = sum_reference(a, M);
    double sum = 0.0;
    for (int i = l; i < q.slices * kSliceNW; i += 64) {
      const float mi = part[i / kSliceNW].m[i % kSliceNW];
      if (mi > kNone) sum += (double)part[i / kSliceNW].sum[i % kSliceNW] * exp(sum_reference(a, mi) - top);
    }
    sum = wave_sum(sum);
    if (l == 0) {
      row_sum = sum;
      row_m = M;
    }
  }
  if (wave_id() == 0) {  // the lists: two slices per lane
    const int l = lane_id();
    const auto either = [](uint32_t u, uint32_t v) { return u | v; };
    uint32_t n[2] = {0u, 0u}, flags = 0u, over = 0u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (2 * l + j < q.slices) {
        n[j] = (uint32_t)part[2 * l + j].count;
        flags |= (uint32_t)part[2 * l + j].flags;
        over |= part[2 * l + j].count > q.cap ? 1u : 0u;
      }
    }
    flags = wave_reduce(flags, 0u, either);
    over = wave_reduce(over, 0u, either);
    const uint32_t inc = wave_incl_scan(n[0] + n[1]);
    first[2 * l] = inc - n[0] - n[1];
    first[2 * l + 1] = inc - n[1];
    if (l == 63) first[kTopSlices] = inc;
    if (l == 0) {
      row_flags = flags;
      row_over = over;
    }
  }
  __syncthreads();
  const uint32_t total = first[kTopSlices];
  const float M = row_m, t = part[0].t;
  const int k = row_k(a, r);
  const int status = top_status(row_flags, M, k);
  float lse = 0.0f;
  if (threadIdx.x == 0 && status == DSPARK_ST_OK) lse = (float)(sum_reference(a, M) + log(row_sum));
  int n = 0;
  uint32_t key[kTopPer], id[kTopPer];
  float v[kTopPer];
#pragma unroll
  for (int j = 0; j < kTopPer; ++j) {
    key[j] = 0u;
    id[j] = 0u;
    v[j] = 0.0f;
  }
  TopCut cut{0xffffffffu, 0u};
  if (status == DSPARK_ST_OK && k > 0) {
    if (row_over || total > (uint32_t)(kTopPer * 64 * NWV) || (total < (uint32_t)k && t > -3.4028235e38f)) {
      n = top_from_memory<DT, NWV>(a, r, k, sh);  // (uniform)
      top_row_out(a, r, status, n, lse);
      return;
    }
    n = total < (uint32_t)k ? (int)total : k;
    // this thread's candidates: neighbours in id order
    const int per = (int)((total + 64 * NWV - 1) / (64 * NWV));
    const typename Cand<DT>::T* lists = static_cast<const typename Cand<DT>::T*>(q.cand) + r * q.slices * q.cap;
    uint32_t at[kTopPer];
    typename Cand<DT>::T e[kTopPer];
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {  // where they lie
      const uint32_t g = threadIdx.x * (uint32_t)per + (uint32_t)j;
      at[j] = 0xffffffffu;
      if (j < per && g < total) {
        int lo = 0, hi = q.slices - 1;  // the last slice that starts at or before g
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (first[mid] <= g) lo = mid;
          else hi = mid - 1;
        }
        id[j] = (uint32_t)lo;
        at[j] = (uint32_t)(lo * q.cap) + g - first[lo];
      }
    }
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {  // all loads on their way
      e[j] = typename Cand<DT>::T{};
      if (at[j] != 0xffffffffu) e[j] = lists[at[j]];
    }
#pragma unroll
    for (int j = 0; j < kTopPer; ++j) {
      if (at[j] != 0xffffffffu) {
        v[j] = Cand<DT>::value(e[j]);
        id[j] = id[j] * (uint32_t)kTopSlice + (uint32_t)Cand<DT>::place(e[j]);
        key[j] = top_key<DT>(v[j]);
      }
    }
    if (n > 0) cut = top_cut<NWV>(key, top_key<DT>(t), top_key<DT>(M), (uint32_t)n, sh);
  }
  top_write<NWV>(a, r, key, cut, n, sh, [&](int j) { return (int32_t)id[j]; }, [&](int j) { return v[j]; });
  top_row_out(a, r, status, n, lse);
}

}  // namespace dspark
